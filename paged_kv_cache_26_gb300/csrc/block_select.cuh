// Block-sparse decode (sm_103a): bounds of each block's keys, the choice of the
// blocks whose bounds promise the largest logits, and decode attention over a
// list of blocks.
//
// Bounds.  For the keys K_t of a (block, KV head), q . K_t <= sum_d max(q_d u_d,
// q_d l_d) with u, l their largest and smallest value in every dim.  u and l are
// held in 8 bits, u rounded up and l down, with one float32 scale s: 2 D + 4 bytes
// where the block's K and V have 64 D.  The query is rounded to 8 bits too (c, scale
// r), so that the sum over dims is one of whole numbers below 2^24, exact in
// float32 as in any other evaluation, and the score, two float32 products
// (sum * s) * r, is the same number wherever it is computed: the choice has no
// rounding of its own, and ties go to the lowest block.
#pragma once

#include <cfloat>

#include "int4_cache.cuh"
#include "paged_kv_kernels.cuh"

namespace pkv {

// ===================================================================== bounds of keys

constexpr int kBoundWarps = 4;

struct BoundArgs {
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_offsets;  // [B + 1], or null: one new token of each sequence
  int8_t* bounds;            // [num_blocks][Hkv][2][D]
  float* scales;             // [num_blocks][Hkv]
  int32_t num_seqs, num_kv_heads, num_blocks, max_blocks, num_tokens;
  int64_t num_items;         // upper limit of the (sequence, block) pairs
};

// Last b in [0, n) with start(b) <= x, where start rises with b and start(0) <= x:
// the warp looks at 32 candidates at once, so a batch of 1024 takes two rounds.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int64_t x, int lane, F&& start) {
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const bool below = at < len && start(lo + at) <= x;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

// One warp per (block, KV head): 16 lanes (8 at D = 64) across a row, 16 bytes
// each, the rows split over the rest of the warp, so a tile is read whole in
// 4 (D = 64) or 8 loads a lane, all in flight.  Extremes are exact on packed pairs.
// Bound by the bytes of the tiles where they are many (the blocks of 8 prompts, 18,000
// tokens, 8 heads, D = 128: 39.5 MB in 10.0 us, 3.9 TB/s with launch and ramp; 7.8 from
// L2), by the chain offsets, table, tile, result where they are few (61 sequences: 3.1
// us).  With eight CTAs asked for on an SM the compiler keeps all eight loads together
// (without it, or with twelve, 12.4 us; eight warps a CTA 10.3).
template <typename T, int D>
__global__ void __launch_bounds__(kBoundWarps * 32, 8) update_bounds_kernel(const BoundArgs a) {
  constexpr int kLanes = D / 8;             // lanes of a row
  constexpr int kRows = 32 / kLanes;        // rows of a load: 2 or 4
  constexpr int kLoads = kBlockSize / kRows;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kBoundWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t item = unit / a.num_kv_heads;
  const int h = static_cast<int>(unit - item * a.num_kv_heads);
  if (item >= a.num_items) return;

  // Items of sequence b start at q_offsets[b] / 16 + 2 b, which leaves room for
  // the blocks that n tokens can touch, at most n / 16 + 2.
  int b, j;
  int ctx;
  if (a.q_offsets) {
    b = warp_search(a.num_seqs, item, lane, [&](int s) {
      return static_cast<int64_t>(__ldg(a.q_offsets + s)) / kBlockSize + 2 * static_cast<int64_t>(s);
    });
    const int o0 = __ldg(a.q_offsets + b), o1 = __ldg(a.q_offsets + b + 1), n = o1 - o0;
    ctx = clamped_context(a.context_lens, b, a.max_blocks, lane == 0 && h == 0);
    // (The last offset tells of sequences that have no items for lack of room.)
    if (unit == 0 && lane == 0 && __ldg(a.q_offsets + a.num_seqs) > a.num_tokens) flag_error(kErrOffsets);
    if (o0 < 0 || o1 < o0 || o1 > a.num_tokens) {
      if (lane == 0) flag_error(kErrOffsets);
      return;
    }
    if (n == 0 || item < o0 / kBlockSize + 2 * static_cast<int64_t>(b)) return;
    const int64_t first = max(ctx - n, 0) / kBlockSize;
    const int64_t at = first + (item - (o0 / kBlockSize + 2 * static_cast<int64_t>(b)));
    if (at >= (ctx + kBlockSize - 1) / kBlockSize) return;
    j = static_cast<int>(at);
  } else {
    b = static_cast<int>(item);
    ctx = clamped_context(a.context_lens, b, a.max_blocks, lane == 0 && h == 0);
    if (ctx == 0) return;
    j = (ctx - 1) / kBlockSize;
  }
  const int phys = __ldg(a.block_tables + static_cast<int64_t>(b) * a.max_blocks + j);
  if (phys < 0 || phys >= a.num_blocks) {
    if (lane == 0) flag_error(kErrBlockId);
    return;
  }
  const int valid = min(kBlockSize, ctx - j * kBlockSize);
  const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + h;
  // A row past the end gives way to the last valid one, which changes no extreme.
  const uint4* src = static_cast<const uint4*>(a.k_cache) + tile * (kBlockSize * kLanes) + lane % kLanes;
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) v[i] = src[min(i * kRows + lane / kLanes, valid - 1) * kLanes];
  uint4 hi = v[0], lo = v[0];
#pragma unroll
  for (int i = 1; i < kLoads; ++i) {
    hi = make_uint4(max2<T>(hi.x, v[i].x), max2<T>(hi.y, v[i].y), max2<T>(hi.z, v[i].z), max2<T>(hi.w, v[i].w));
    lo = make_uint4(min2<T>(lo.x, v[i].x), min2<T>(lo.y, v[i].y), min2<T>(lo.z, v[i].z), min2<T>(lo.w, v[i].w));
  }
#pragma unroll
  for (int o = 16; o >= kLanes; o >>= 1) {
    hi = make_uint4(max2<T>(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o)),
                    max2<T>(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o)),
                    max2<T>(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o)),
                    max2<T>(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o)));
    lo = make_uint4(min2<T>(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o)),
                    min2<T>(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o)),
                    min2<T>(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o)),
                    min2<T>(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o)));
  }
  float u[8], l[8], top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<T>(word_of(hi, i)), y = unpack2<T>(word_of(lo, i));
    u[2 * i] = x.x;
    u[2 * i + 1] = x.y;
    l[2 * i] = y.x;
    l[2 * i + 1] = y.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = fmaxf(fabsf(u[i]), fabsf(l[i]));
    finite = finite && fabsf(u[i]) < INFINITY && fabsf(l[i]) < INFINITY;  // false for NaN
    top = fmaxf(top, m);
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  finite = __all_sync(0xffffffffu, finite);
  const float s = finite ? __fmul_rn(top, 1.f / 127.f) : INFINITY;
  uint32_t cu[2] = {0, 0}, cl[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int x = 127, y = -127;
    if (finite) {
      x = s > 0.f ? static_cast<int>(fminf(fmaxf(ceilf(__fdiv_rn(u[i], s)), -127.f), 127.f)) : 0;
      y = s > 0.f ? static_cast<int>(fminf(fmaxf(floorf(__fdiv_rn(l[i], s)), -127.f), 127.f)) : 0;
    }
    cu[i >> 2] |= static_cast<uint32_t>(x & 255) << (8 * (i & 3));
    cl[i >> 2] |= static_cast<uint32_t>(y & 255) << (8 * (i & 3));
  }
  if (lane < kLanes) {
    uint2* dst = reinterpret_cast<uint2*>(a.bounds + tile * (2 * D)) + lane;
    dst[0] = make_uint2(cu[0], cu[1]);
    dst[kLanes] = make_uint2(cl[0], cl[1]);
    if (lane == 0) a.scales[tile] = s;
  }
}

// ===================================================================== scores

struct SelectArgs {
  const void* q;             // T[B][Hq][D]
  const int8_t* bounds;
  const float* scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint32_t* keys;            // workspace: [B][Hkv][max_blocks] ordered scores
  int32_t* selected;         // [B][Hkv][num_selected]
  int32_t num_seqs, num_q_heads, num_kv_heads, group, num_blocks, max_blocks;
  int32_t num_selected, sink, recent;
};

constexpr int kScoreThreads = 128;  // of a CTA, a block each; of one that chooses too:
constexpr int kWholeThreads = 256;
constexpr int kScoreCtas = 4096;    // CTAs for the ranges of all tables, about
// Two on each SM (64 KB of rows, at most 107 registers).  A number, not the device's SMs, so
// that the size of the workspace does not depend on which device is current.
constexpr int kWholeUnits = 2 * 152;

// Unsigned numbers in the order of the floats (there is no -0 among them); NaN as
// +infinity.
__device__ __forceinline__ uint32_t ordered_key(float x) {
  const uint32_t u = x != x ? 0x7f800000u : __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// --------------------------------------------------------------------- choice among keys

constexpr int kSelectThreads = 1024;  // of a CTA; 256 for tables of up to 2,048 blocks (below)
constexpr int kSelectRun = 8;         // keys that a thread holds in registers, at most
constexpr int kSelectCached = 32768;  // keys of longer contexts held in shared memory (132 KB); past it they are read again
// A word in 33 is left out, so that threads on runs of neighbouring keys meet different
// banks.
__host__ __device__ constexpr int select_place(int i) { return i + (i >> 5); }

// One CTA per (sequence, KV head): a radix selection finds the smallest chosen key
// and how many of its equals are chosen, then one pass writes the chosen blocks in
// rising order: a thread takes a run of neighbouring blocks and learns from one
// scan how many lie before it.  Runs of up to kSelectRun blocks stay in registers; a
// thread holds so many, so the CTA is as small as the table allows, 256 threads up to
// 2,048 blocks (its barriers cost less, and 1,024 threads of 64 registers are alone on
// their SM: 32 x 8 choices were then 2.5 us slower than with keys in shared memory).  Bound by the chain of loads, up to four rounds of counting with two
// barriers each, and the scan: about 6 us for 8,192 blocks (keys in shared memory 9); the
// keys are few bytes.  (Scores and choice in one kernel, a cluster a (sequence, KV head):
// 40 us against 28, as both then were, for the whole step of 131,072 tokens.)
template <int kThreads, bool kRegs, typename Fresh>
__device__ __forceinline__ void choose_blocks(const Fresh& fresh, int nb, uint32_t left, int32_t* out) {
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) uint32_t s_hist[4][256];
  __shared__ uint32_t s_state[3];        // prefix found so far, how many still to choose among its bin, all of it
  __shared__ uint32_t s_warp[2][33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (nb + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, nb), i1 = min(i0 + per, nb);
  const bool cached = nb <= kSelectCached;
  uint32_t run[kSelectRun];
  if (kRegs) {
#pragma unroll
    for (int j = 0; j < kSelectRun; ++j) run[j] = i0 + j < i1 ? fresh(i0 + j) : 0;
  } else if (cached) {
#pragma unroll 8
    for (int i = tid; i < nb; i += kThreads) s_key[select_place(i)] = fresh(i);
  }
#pragma unroll
  for (int i = tid; i < 1024; i += kThreads) s_hist[i >> 8][i & 255] = 0;
  __syncthreads();
  // f(block, key) for this thread's run, and for any share of the blocks.
  auto each_in_run = [&](auto&& f) {
    if (kRegs) {
#pragma unroll
      for (int j = 0; j < kSelectRun; ++j)
        if (i0 + j < i1) f(i0 + j, run[j]);
    } else {
      for (int i = i0; i < i1; ++i) f(i, cached ? s_key[select_place(i)] : fresh(i));
    }
  };
  auto each = [&](auto&& f) {
    if (kRegs)
      each_in_run(f);
    else
      for (int i = tid; i < nb; i += kThreads) f(i, cached ? s_key[select_place(i)] : fresh(i));
  };
  uint32_t prefix = 0;
  int shift = 24;
  for (;; shift -= 8) {
    uint32_t* hist = s_hist[shift >> 3];
    each([&](int, uint32_t k) {
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    });
    __syncthreads();
    if (warp == 0) {
      // Lane l counts bins 255 - 8 l downwards; the bin where the count reaches `left`.
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - 8 * lane - i];
        sum += c[i];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
      if (before < left && before + sum >= left) {
        int bin = 255 - 8 * lane;
        uint32_t in_bin = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          in_bin = c[i];
          if (before + c[i] >= left) break;
          before += c[i];
          --bin;
        }
        s_state[0] = prefix << 8 | static_cast<uint32_t>(bin);
        s_state[1] = left - before;
        s_state[2] = in_bin == left - before;
      }
    }
    __syncthreads();
    prefix = s_state[0];
    left = s_state[1];
    if (shift == 0 || s_state[2]) break;  // (a bin chosen whole needs no further digits)
  }
  // By their digits down to `shift`: all keys above `prefix`, and the first `left` of
  // those equal to it.
  uint32_t above = 0, equal = 0;
  each_in_run([&](int, uint32_t k) {
    above += (k >> shift) > prefix;
    equal += (k >> shift) == prefix;
  });
  uint32_t sa = above, se = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t va = __shfl_up_sync(0xffffffffu, sa, o), ve = __shfl_up_sync(0xffffffffu, se, o);
    if (lane >= o) {
      sa += va;
      se += ve;
    }
  }
  if (lane == 31) {
    s_warp[0][warp] = sa;
    s_warp[1][warp] = se;
  }
  __syncthreads();
  // Every warp sums the warps before it.
  const uint32_t wa = lane < warp ? s_warp[0][lane] : 0, we = lane < warp ? s_warp[1][lane] : 0;
  sa += __reduce_add_sync(0xffffffffu, wa) - above;  // keys above / equal before this thread's run
  se += __reduce_add_sync(0xffffffffu, we) - equal;
  each_in_run([&](int i, uint32_t k) {
    const uint32_t at = sa + min(se, left);
    if ((k >> shift) > prefix) {
      out[at] = i;
      ++sa;
    } else if ((k >> shift) == prefix) {
      if (se < left) out[at] = i;
      ++se;
    }
  });
}

// --------------------------------------------------------------------- scores

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A CTA scores ranges of 128 blocks of one (sequence, KV head) for its G >= group heads, a
// warp 32 of each.
// The warp starts the copies of all its rows of bounds (2 D bytes each) at once, 8 KB at
// D = 128, without a register for them; the query's codes are made while they come.
// max(4, G) lanes share a row, 16 bytes at a time, upper bounds in its first half; they
// keep the codes for their bytes in registers, the positive ones against the upper
// bounds, the negative ones against the lower, as four-way byte products.  The G sums are
// then folded over the lanes, half of the sums going either way in each exchange, after
// which a lane holds one head's.
// Bound by the latency of table, bounds and their bytes: with the choice after it, 32
// sequences of 8,192 to 32,768 tokens, 8 KV heads, G = 4, D = 128 (85 MB) take 25.6 us,
// 131,072 tokens of one sequence, G = 8 (17 MB) 13.3.  (Loads through registers, eight a
// lane under way, 16 lanes a row: 37.7 and 21.8 with the choice of that time; four lanes
// a row and loads through registers: 6 us slower than copies at G = 4, as fewer CTAs fit.
// The products as s8 tensor products: no gain over byte products.)
//
// kWhole: the table has no more blocks than the CTA threads, and the CTA chooses as well.
template <typename T, int D, int G, bool kWhole>
__global__ void __launch_bounds__(kWhole ? kWholeThreads : kScoreThreads) score_blocks_kernel(const SelectArgs a) {
  constexpr int kLanes = G == 8 ? 8 : 4;
  constexpr int kPieces = 2 * D / 16;                // 16-byte pieces of a row
  constexpr int kTurns = kPieces / kLanes;
  constexpr int kRows = 32 / kLanes;                 // blocks of a warp's step
  constexpr int kThreads = kWhole ? kWholeThreads : kScoreThreads;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(128) uint4 s_rows[];   // [kThreads][kPieces]
  __shared__ uint32_t s_keys[kWhole ? kThreads : 1];
  __shared__ __align__(16) int8_t s_code[G][2 * D];  // the positive codes, against upper bounds; the negative ones
  __shared__ float s_scale[G];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The heads of a range side by side, so that their pieces of a block, neighbours in
  // memory, are read at about the same time.
  const int h = blockIdx.x % a.num_kv_heads, b = blockIdx.y;
  int first = blockIdx.x / a.num_kv_heads * kThreads;  // of the CTA's blocks
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks;
  int phys = first + threadIdx.x < a.max_blocks ? __ldg(table + first + threadIdx.x) : -1;  // this lane's block
  constexpr int kVals = D / 32, kHeads = (G + kWarps - 1) / kWarps;  // values of a lane, heads of a warp
  float x[kHeads][kVals];
#pragma unroll
  for (int n = 0; n < kHeads; ++n) {
    const int g = warp + n * kWarps;
    const T* q = static_cast<const T*>(a.q) + (static_cast<int64_t>(b) * a.num_q_heads + h * a.group + g) * D;
#pragma unroll
    for (int i = 0; i < kVals; ++i) x[n][i] = g < a.group ? static_cast<float>(q[lane * kVals + i]) : 0.f;
  }
  const int ctx = clamped_context(a.context_lens, b, a.max_blocks, threadIdx.x == 0 && blockIdx.x == 0);
  const int nb = (ctx + kBlockSize - 1) / kBlockSize;
  int32_t* out = a.selected + (static_cast<int64_t>(b) * a.num_kv_heads + h) * a.num_selected;
  if (nb <= a.num_selected) {                        // all are chosen, without scores
    if (kWhole)
      for (int i = threadIdx.x; i < a.num_selected; i += kThreads) out[i] = i < nb ? i : -1;
    return;
  }
  if (first >= nb) return;
  uint4* rows = s_rows + warp * 32 * kPieces;
  // In odd rows the halves of 64 bytes change places: four lanes a row meet all banks.
  auto place = [](int r, int piece) { return r * kPieces + (piece ^ ((r & 1) << 2)); };
  float my_step;                                     // the scale of this lane's block
  auto start_copies = [&]() {
    if (first + static_cast<int>(threadIdx.x) >= nb) {
      phys = -1;
    } else if (phys < 0 || phys >= a.num_blocks) {
      if (h == 0) flag_error(kErrBlockId);
      phys = -1;
    }
    // Without a block: a scale of 0, whatever lies in the row.
    my_step = phys >= 0 ? __ldg(a.scales + static_cast<int64_t>(phys) * a.num_kv_heads + h) : 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = i * (32 / kPieces) + lane / kPieces, piece = lane % kPieces;
      const int p = __shfl_sync(0xffffffffu, phys, r);
      if (p >= 0)
        copy_async16(smem_u32(rows + place(r, piece)),
                     a.bounds + (static_cast<int64_t>(p) * a.num_kv_heads + h) * (2 * D) + 16 * piece);
    }
  };
  start_copies();
#pragma unroll
  for (int n = 0; n < kHeads; ++n) {
    const int g = warp + n * kWarps;
    if (g >= G) break;
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      finite = finite && fabsf(x[n][i]) < INFINITY;
      top = fmaxf(top, fabsf(x[n][i]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    finite = __all_sync(0xffffffffu, finite);
    // A query that is not finite has no codes and an infinite scale: 0 times that, a NaN,
    // is a score of +infinity for every block.
    const float s = finite ? __fmul_rn(top, 1.f / 127.f) : INFINITY;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int c = finite && s > 0.f ? static_cast<int>(rintf(__fdiv_rn(x[n][i], s))) : 0;
      s_code[g][lane * kVals + i] = static_cast<int8_t>(max(c, 0));
      s_code[g][D + lane * kVals + i] = static_cast<int8_t>(min(c, 0));
    }
    if (lane == 0) s_scale[g] = s;
  }
  __syncthreads();
  const int sub = lane % kLanes, grp = lane / kLanes;
  int32_t code[G][kTurns][4];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      const int4 c = *reinterpret_cast<const int4*>(&s_code[g][16 * (t * kLanes + sub)]);
      code[g][t][0] = c.x;
      code[g][t][1] = c.y;
      code[g][t][2] = c.z;
      code[g][t][3] = c.w;
    }
  // After the exchanges below, a lane's sum is of this head.
  int head = 0;
#pragma unroll
  for (int n = G / 2, o = 1; n > 0; n /= 2, o *= 2)
    if (lane & o) head += n;
  const float head_scale = s_scale[head];
  uint32_t* keys = kWhole ? s_keys : a.keys + (static_cast<int64_t>(b) * a.num_kv_heads + h) * a.max_blocks;
  for (;;) {
    const int mine = nb - first - warp * 32;         // blocks of this warp, or more
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (mine > 0) {
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += kRows) {
        const int r = r0 + grp;
        int32_t dot[G];
#pragma unroll
        for (int g = 0; g < G; ++g) dot[g] = 0;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          const uint4 e = rows[place(r, t * kLanes + sub)];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            dot[g] = __dp4a(code[g][t][0], static_cast<int32_t>(e.x), dot[g]);
            dot[g] = __dp4a(code[g][t][1], static_cast<int32_t>(e.y), dot[g]);
            dot[g] = __dp4a(code[g][t][2], static_cast<int32_t>(e.z), dot[g]);
            dot[g] = __dp4a(code[g][t][3], static_cast<int32_t>(e.w), dot[g]);
          }
        }
        // Exchange halves while there are several sums, then add.
#pragma unroll
        for (int o = 1, n = G; o < kLanes; o *= 2, n = n > 1 ? n / 2 : 1) {
          if (n > 1) {
            const bool odd = lane & o;
#pragma unroll
            for (int g = 0; g < n / 2; ++g) {
              const int32_t give = odd ? dot[g] : dot[g + n / 2];
              const int32_t keep = odd ? dot[g + n / 2] : dot[g];
              dot[g] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          } else {
            dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
          }
        }
        // A NaN (0 times an infinite scale, of the bounds or the query) is +infinity, as in
        // ordered_key.
        // Adding 0 makes a product that underflowed to -0 the equal of +0.
        const float step = __shfl_sync(0xffffffffu, my_step, r);
        float score = __fadd_rn(__fmul_rn(__fmul_rn(static_cast<float>(dot[0]), step), head_scale), 0.f);
        if (head >= a.group) score = -INFINITY;
        uint32_t key = ordered_key(score);
#pragma unroll
        for (int m = 1; m < G; m *= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, m));
        if (sub == 0 && r < mine) keys[first + warp * 32 + r] = key;
      }
    }
    first += gridDim.x / a.num_kv_heads * kThreads;
    if (kWhole || first >= nb) break;
    __syncwarp();                                    // the rows have been read
    phys = first + threadIdx.x < a.max_blocks ? __ldg(table + first + threadIdx.x) : -1;
    start_copies();
  }
  if constexpr (kWhole) {
    __syncthreads();
    auto fresh = [&](int i) { return i < a.sink || i >= nb - a.recent ? 0xffffffffu : s_keys[i]; };
    choose_blocks<kThreads, true>(fresh, nb, static_cast<uint32_t>(a.num_selected), out);
  }
}

// ===================================================================== choice

template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_blocks_kernel(const SelectArgs a) {
  const int h = blockIdx.x, b = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ctx = clamped_context(a.context_lens, b, a.max_blocks, false);
  const int nb = (ctx + kBlockSize - 1) / kBlockSize;
  const int64_t unit = static_cast<int64_t>(b) * a.num_kv_heads + h;
  int32_t* out = a.selected + unit * a.num_selected;
  if (nb <= a.num_selected) {
    for (int i = threadIdx.x; i < a.num_selected; i += kThreads) out[i] = i < nb ? i : -1;
    return;
  }
  const uint32_t* keys = a.keys + unit * a.max_blocks;
  // The blocks always kept rank above every score.
  auto fresh = [&](int i) { return i < a.sink || i >= nb - a.recent ? 0xffffffffu : __ldcg(keys + i); };
  if (kThreads < kSelectThreads || nb <= kSelectRun * kThreads)
    choose_blocks<kThreads, true>(fresh, nb, static_cast<uint32_t>(a.num_selected), out);
  else
    choose_blocks<kThreads, false>(fresh, nb, static_cast<uint32_t>(a.num_selected), out);
}

// ===================================================================== attention over chosen blocks

constexpr int kSparseWarps = 4;
constexpr int kMaxSparseCluster = 16;

template <int D>
struct SparseShape {
  static constexpr int kStageBytes = TileShape<D>::kStageBytes;  // K and V of a block
  static constexpr int kStages = D == 128 ? 3 : 6;               // 24 KB in flight a warp
  static constexpr int kRing = kSparseWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRing + 1024;
  static_assert((kSparseWarps + 1) * kMaxGroup * (D + 2) * 4 <= kRing, "the merge reuses the ring");
};

// A cluster of CTAs per (sequence, KV head), a CTA of four warps with rings of
// their own (24 KB each, two CTAs an SM).  Warp w of the cluster's W takes entries
// w, w + W, ... of the list, one 16-token block a step with the math of the decode
// kernels; the warps' partial results meet in shared memory, the CTAs' in
// distributed shared memory, so that there is neither workspace nor second launch.
// Bound by the K and V bytes for large batches (32 sequences x 8 KV heads x 128 blocks:
// 268 MB in 45 us, 5.9 TB/s), by the chain list, table, tiles, merge for small ones.
template <typename T, int D>
__global__ void __launch_bounds__(kSparseWarps * 32, 2)
    decode_sparse_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const DecodeArgs args, const int32_t* __restrict__ selected, int32_t num_selected,
                         int32_t cluster) {
  using Shape = SparseShape<D>;
  constexpr int NST = Shape::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kSparseWarps][NST];
  __shared__ int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;  // the cluster spans x
  const int g = args.group;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kSparseWarps; ++w)
      for (int s = 0; s < NST; ++s) mbar_init(smem_u32(&bars[w][s]), 1);
    s_abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int ctx = clamped_context(args.context_lens, b, args.max_blocks, threadIdx.x == 0 && rank == 0 && kvh == 0);
  const int nblk = (ctx + kBlockSize - 1) / kBlockSize;
  const int32_t* list = selected + (static_cast<int64_t>(b) * args.num_kv_heads + kvh) * num_selected;
  const int32_t* table = args.block_tables + static_cast<int64_t>(b) * args.max_blocks;
  const int stride = cluster * kSparseWarps, me = rank * kSparseWarps + warp;
  const uint32_t ring = smem_u32(smem + warp * NST * Shape::kStageBytes);
  const uint64_t policy = l2_evict_first_policy();

  WarpAttn<T, D> at;
  at.reset();
  // The smallest finite reference, so that logits of -infinity weigh 0 beside others
  // instead of giving NaN; -infinity is left to partial results without a block.
  at.m0 = at.m1 = -FLT_MAX;
  at.load_q(static_cast<const T*>(args.q) + (static_cast<int64_t>(b) * args.num_q_heads + kvh * g) * D, g, lane);

  // Windows of 32 entries: lane i holds the row and the valid tokens of one.
  bool ok = true;
  int issued = 0, used = 0;  // blocks of this warp so far
  for (int base = me; base < num_selected && ok; base += 32 * stride) {
    const int e = base + lane * stride;
    int valid = 0, row = 0;
    if (e < num_selected) {
      const int j = __ldg(list + e);
      if (j >= nblk) flag_error(kErrSelected);
      if (j >= 0 && j < nblk) {
        valid = min(kBlockSize, ctx - j * kBlockSize);
        row = tile_row(__ldg(table + j), kvh, args);
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, valid > 0);
    uint32_t ahead = todo;
    // Fill the ring, then refill each stage once it has been used.
    auto issue = [&]() {
      const int from = __ffs(ahead) - 1;
      ahead &= ahead - 1;
      const int r = __shfl_sync(0xffffffffu, row, from);
      if (lane == 0)
        issue_block<D>(ring + (issued % NST) * Shape::kStageBytes, smem_u32(&bars[warp][issued % NST]), &tmap_k, &tmap_v,
                       r, policy);
      ++issued;
    };
    while (ahead && issued - used < NST) issue();
    while (todo && ok) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      const int n = __shfl_sync(0xffffffffu, valid, from);
      const int st = used % NST;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), (used / NST) & 1));
      if (!ok) break;
      const uint8_t* ks = smem + warp * NST * Shape::kStageBytes + st * Shape::kStageBytes;
      at.block(ks, ks + TileShape<D>::kTileBytes, n, args.scale_log2, lane);
      __syncwarp();
      ++used;
      if (ahead) issue();
    }
  }
  if (!ok) {
    s_abort = 1;  // (the wait has flagged it); copies in flight may not outlive the CTA
    for (; used < issued; ++used) mbar_wait(smem_u32(&bars[warp][used % NST]), (used / NST) & 1);
  }
  at.finish_sums();
  __syncthreads();  // rings drained: reused for the merge

  float* red_o = reinterpret_cast<float*>(smem);            // [warps][8][D], then the CTA's [8][D]
  float* red_m = red_o + (kSparseWarps + 1) * kMaxGroup * D;  // [warps + 1][8]
  float* red_l = red_m + (kSparseWarps + 1) * kMaxGroup;
  {
    const int gid = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hd = 2 * c + e;
      if (gid == 0) {
        red_m[warp * kMaxGroup + hd] = used == 0 ? -INFINITY : e ? at.m1 : at.m0;
        red_l[warp * kMaxGroup + hd] = e ? at.l1 : at.l0;
      }
      float* dst = red_o + (warp * kMaxGroup + hd) * D;
#pragma unroll
      for (int kk = 0; kk < WarpAttn<T, D>::kChunks; ++kk) {
        float v[8];
        at.chunk_values(e, kk, 1.0f, v);
        float4* d4 = reinterpret_cast<float4*>(dst + WarpAttn<T, D>::chunk_dim(lane, kk));
        d4[0] = make_float4(v[0], v[1], v[2], v[3]);
        d4[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
  __syncthreads();
  // Weighted sum over `n` partial results of this row, 2^(m - max) each (a partial
  // without a block has m = -infinity and weight 0).
  constexpr int kQuads = D / 4;
  float* cta_o = red_o + kSparseWarps * kMaxGroup * D;
  for (int idx = threadIdx.x; idx < g * kQuads; idx += kSparseWarps * 32) {
    const int r = idx / kQuads, d4 = (idx - r * kQuads) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) M = fmaxf(M, red_m[w * kMaxGroup + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
      const float mw = red_m[w * kMaxGroup + r];
      const float wt = mw == -INFINITY && red_l[w * kMaxGroup + r] == 0.f ? 0.f : exp2f(mw - M);
      L += red_l[w * kMaxGroup + r] * wt;
      const float4 v = *reinterpret_cast<const float4*>(red_o + (w * kMaxGroup + r) * D + d4);
      o.x += v.x * wt;
      o.y += v.y * wt;
      o.z += v.z * wt;
      o.w += v.w * wt;
    }
    *reinterpret_cast<float4*>(cta_o + r * D + d4) = o;
    if (d4 == 0) {
      red_m[kSparseWarps * kMaxGroup + r] = M;
      red_l[kSparseWarps * kMaxGroup + r] = L;
    }
  }
  if (cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  const bool aborted = *reinterpret_cast<volatile int*>(&s_abort) != 0;
  // The cluster's CTAs share the output's quads between them.
  auto peer = [&](const float* p, int r) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(r));
    return addr;
  };
  for (int idx = rank * (kSparseWarps * 32) + threadIdx.x; idx < g * kQuads; idx += stride * 32) {
    const int r = idx / kQuads, d4 = (idx - r * kQuads) * 4;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ms[kMaxSparseCluster], ls[kMaxSparseCluster];
#pragma unroll
    for (int c = 0; c < kMaxSparseCluster; ++c) {
      ms[c] = -INFINITY;
      ls[c] = 0.f;
      if (c < cluster) {
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ms[c]) : "r"(peer(red_m + kSparseWarps * kMaxGroup + r, c)));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ls[c]) : "r"(peer(red_l + kSparseWarps * kMaxGroup + r, c)));
      }
      M = fmaxf(M, ms[c]);
    }
#pragma unroll
    for (int c = 0; c < kMaxSparseCluster; ++c) {
      if (c >= cluster) break;
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(peer(cta_o + r * D + d4, c)));
      const float wt = ms[c] == -INFINITY && ls[c] == 0.f ? 0.f : exp2f(ms[c] - M);
      L += ls[c] * wt;
      o.x += v.x * wt;
      o.y += v.y * wt;
      o.z += v.z * wt;
      o.w += v.w * wt;
    }
    if (aborted) continue;
    // No block: a zero row; nothing but logits of -infinity: NaN, as softmax is (a NaN stays one).
    const float inv = L != 0.f ? 1.0f / L : M == -INFINITY ? 0.f : __int_as_float(0x7fffffff);
    uint2 pk;
    pk.x = pack2<T>(o.x * inv, o.y * inv);
    pk.y = pack2<T>(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(args.out) +
                              (static_cast<int64_t>(b) * args.num_q_heads + kvh * g + r) * D + d4) = pk;
  }
  // No CTA may leave while another still reads its shared memory.
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace pkv
