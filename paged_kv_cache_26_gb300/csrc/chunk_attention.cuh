// Attention of chunks of new tokens over a paged cache (sm_103a): causal, ragged,
// any number of new tokens a sequence, on the fifth-generation tensor cores.
//
// A work unit is up to 256 query rows of one (sequence, KV head): the rows of
// consecutive new tokens with their group of query heads packed (row = token * g +
// head), as two tiles A and B of 128 rows (128 / g whole tokens each).  It walks its
// keys in tiles of 128 tokens (eight blocks):
//   S = Q K^T        M = 128 rows, N = 128 keys, from shared memory into TMEM
//   P = 2^(S c - m)  in registers, one thread a row; m, the row's reference, moves
//                    only when a score passes it by 2^8, so O is rarely rescaled, and
//                    the weights need not wait for the tile's maximum
//   O += P V         P from TMEM (over S's columns), O in TMEM, fp32
// The tensor pipe alternates between the tiles, PV_A S_A' PV_B S_B', so that the
// softmax of one tile runs under the products of the other.  Either tile has an
// issuing warp of its own: an MMA waits in its thread until the tensor pipe can
// queue it, and a barrier that is ready costs 100 to 200 cycles, which the pipe would
// spend idle behind a single thread (438 us against 361, at the size below).
//
// Bound by the tensor pipe at D = 128: 2,048 new tokens after 14,000, 32 query and 8 KV
// heads, bf16, 315 to 326 us (1.55 to 1.60 PFLOP/s of the measured 1.87; the tensor pipe is
// busy for 75 % of the main kernel, the pipe of the exponentials for 37 %).  D = 64 258 us,
// where a key costs half the products and the same exponentials: tensor pipe and
// exponentials 41 % busy each, issue 47 %, so what bounds it is the chain scores,
// softmax, product, which two tiles do not fill.  2,048 tokens after 63,001: 1.51 to 1.57 ms
// (1.37 to 1.43 PFLOP/s).  A step of 64 single tokens of 2,000 to 4,000 tokens each 136 us:
// four of a tile's 128 rows hold a token's group, and K and V bound it.
//
// Work is divided by keys, not by units: the units' keys (plus a fixed amount for
// a unit's start and end) form one line which is cut into equal parts, one per
// CTA, one CTA per SM.  A part begins and ends inside units; such pieces leave
// unnormalised fp32 partial results that merge_chunk_kernel joins in order.  Every
// cut follows from the lengths alone, by closed sums that each CTA computes for
// itself; nothing is counted or claimed at run time.  Where there are CTAs enough for
// one unit each and all contexts are short, the line counts units and nothing is cut;
// if the tables are too narrow for long contexts, the merge is not launched either.
//
// Values that a row does not attend to may be anything.  Scores there are replaced,
// not weighted.  A weight of 0 would still meet V in the product (0 * NaN = NaN), so
// a warp between TMA and MMA goes over V in the tiles where some row attends to less
// than all: rows past the sequence become zeros, and if a value that later rows
// attend to is not finite, the tile's P V is summed by the softmax threads instead,
// each row its own tokens.
//
// Warps: 0-3 softmax of tile A, 4-7 of tile B, 8 TMA, 9 and 10 MMA of A and B, 11 V.
// Every wait is on a phase at most one ahead of the last completed one: the TMA,
// V and MMA warps go through all tiles in order, a tile that concerns only one of
// the MMA warps included.  Waits give up after kWaitLimitNs.
#pragma once

#include <cfloat>
#include <climits>

#include "paged_kv_kernels.cuh"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kChunkKeys = 128;            // keys of a tile
constexpr int kChunkRows = 256;            // query rows of a unit
constexpr int kChunkThreads = 384;
constexpr int kMaxChunkSeqs = 8192;
constexpr int kChunkPieces = 4;            // pieces known ahead
constexpr int kChunkSteps = 16;            // barriers of steps: more than can be under way (a tile of the ring each)
// Quarters of a tile's weights whose product begins before the others are made: 1 315 us,
// 2 339, 3 361, all at once 348; an arrival for every quarter 346, half a quarter 329.
constexpr int kEarly = 1;
// A unit's start and end (first loads, first softmax, output) in keys, and the least
// number of keys worth a CTA of its own.
constexpr int kUnitKeys = 128;
constexpr int kLeastKeys = 512;
// Units of at most so many keys are not cut where there are CTAs enough for one each:
// partial results and their merge cost more than what they share out.  32/8 heads, D =
// 128: 3 sequences of up to 260 tokens 12.1 us against 23.2, 512 new tokens from 0 14.6
// against 23.2, 16 single tokens of 500 to 1,000 18.3 against 20.9; 2 of 1,000 17.0 against
// 16.5, 2 of 2,000 26.5 against 17.9.  (About 2 us more where only the GPU knows that they
// are short.)
constexpr int kWholeKeys = 1024;
// A row's reference before its first weight: finite, so that logits of -infinity weigh 0
// under it as under any other.  It tells rows without any weight apart, in partial results
// too: one whose visible logits are all -infinity is NaN, as softmax is, one that sees no
// key zero.
constexpr float kLeastRef = -FLT_MAX, kNoKeysRef = -3e38f;

// How a CTA's part begins, for the merge: inside a unit (its first piece is then
// partial result 2 cta) and, `open`, ends inside it too.
struct ChunkCut {
  int32_t cut, open;
  int32_t row0, tokens, kvh;  // the unit's
  int32_t unused[3];
};

struct ChunkArgs {
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_offsets;
  float* part;              // [2 grid][256 * (D + 2)]: O as [D / 4][256 rows] of four dims, then m and l of every row
  ChunkCut* cuts;           // [grid]
  float c2;                 // |scale| * log2(e), at least the smallest float
  int32_t negate;           // scale < 0: S is negated in the product
  int32_t grid;             // CTAs of the main kernel
  int32_t num_tokens, num_seqs, num_q_heads, num_kv_heads, group, max_blocks, num_blocks;
  int32_t tile_tokens;      // tokens of a tile: 128 / group
  // The line may count units instead of keys, so that no cut lies inside one: there are
  // CTAs enough, and the contexts are known to be short (2) or may turn out so (1).
  int32_t whole_units;
};

template <int D>
struct ChunkShape {
  // Tiles lie in swizzled atoms of 8 rows x 64 dims (1 KB).  Queries: the atoms of
  // the first 64 dims, then of the others.  Keys and values: the atoms of 8 tokens
  // side by side, so that a block is one run of shared memory and one TMA box
  // (a box's cost is per instruction: two boxes of 2 KB a block took 32
  // instructions and 3,200 cycles for a K and a V tile).
  static constexpr int kQHalf = 128 * 128;
  static constexpr int kAtom = 1024;
  static constexpr int kGroup = kAtom * (D / 64);            // 8 tokens
  static constexpr int kTileBytes = kChunkKeys * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;           // ring of K and V tiles: 160 KB
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024;
  static constexpr int kSCol = 0, kOCol = 256;               // TMEM: S (and P) 128 columns a tile, then O
  static constexpr int kTmemCols = 512;
  static constexpr int64_t kPart = static_cast<int64_t>(kChunkRows) * (D + 2);  // floats of a partial result
};

// ------------------------------------------------------------------ the line of work

// One sequence's share of the line.
struct ChunkSeq {
  int o0, n, ctx;  // first row, new tokens, context
  int units;       // per KV head
  int before;      // max(ctx - n, 0): keys before the chunk
  bool whole;      // the line counts units
  int64_t line;    // length per KV head

  // Where unit i starts, from the start of its (sequence, KV head).
  __device__ __forceinline__ int64_t start(int i, int tt) const {
    if (whole) return i;
    return static_cast<int64_t>(i) * (before + kUnitKeys) + static_cast<int64_t>(tt) * (static_cast<int64_t>(i) * (i + 1) / 2);
  }
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs& a, int b, bool flag, bool whole) {
  ChunkSeq s;
  const int r0 = __ldg(a.q_offsets + b), r1 = __ldg(a.q_offsets + b + 1);
  s.o0 = min(max(r0, 0), a.num_tokens);
  const int o1 = min(max(r1, 0), a.num_tokens);
  s.n = max(o1 - s.o0, 0);
  if (flag && (r0 < 0 || r1 < r0 || r1 > a.num_tokens)) flag_error(kErrOffsets);
  s.ctx = clamped_context(a.context_lens, b, a.max_blocks, flag);
  const int tt = 2 * a.tile_tokens;
  s.units = (s.n + tt - 1) / tt;
  s.before = max(s.ctx - s.n, 0);
  s.whole = whole;
  s.line = s.whole ? s.units : s.n > 0 ? s.start(s.units - 1, tt) + s.before + s.n + kUnitKeys : 0;
  return s;
}

// What a CTA does of one unit.
struct ChunkPiece {
  int b, kvh;
  int row0;        // first row of q
  int tokens;      // of the unit, 1 .. 2 tile_tokens
  int first;       // position of its first token (negative: the context is shorter than the chunk)
  int ctx;
  int t0, t1;      // key tiles of this piece
  int kt[2];       // key tiles of the unit, for its tiles A and B
  int slot;        // partial result, or -1: the piece is the whole unit
  __device__ __forceinline__ int tiles() const { return max(kt[0], kt[1]); }
  __device__ __forceinline__ int end(int q) const { return min(t1, kt[q]); }
};

// Position on the line, and a walk along it.
struct ChunkWalk {
  ChunkSeq s;
  int b, kvh, unit;
  int64_t unit_at;  // where the unit starts on the line
  int64_t at, stop; // what is left of this CTA's part

  __device__ __forceinline__ int64_t cost(int tt) const {
    if (s.whole) return 1;
    return min(static_cast<int64_t>(unit + 1) * tt, static_cast<int64_t>(s.n)) + s.before + kUnitKeys;
  }
  // The unit at `at`, which lies `rest` into sequence b.
  __device__ __forceinline__ void locate(const ChunkArgs& a, int seq, int64_t rest, bool whole) {
    const int tt = 2 * a.tile_tokens;
    b = seq;
    s = chunk_seq(a, b, false, whole);
    // Quotient and root in float32, corrected by a step or two.
    kvh = min(static_cast<int>(static_cast<float>(rest) / static_cast<float>(s.line)), a.num_kv_heads - 1);
    while (kvh > 0 && kvh * s.line > rest) --kvh;
    while ((kvh + 1) * s.line <= rest) ++kvh;
    rest -= kvh * s.line;
    // start(i) <= rest, i the positive root: 2 rest / (p + sqrt(p^2 + 2 tt rest)).
    const float p = static_cast<float>(s.before + kUnitKeys) + 0.5f * tt, x = static_cast<float>(rest);
    int i = s.whole ? static_cast<int>(rest) : static_cast<int>(2.f * x / (p + sqrtf(p * p + 2.f * tt * x)));
    i = min(max(i, 0), s.units - 1);
    while (i > 0 && s.start(i, tt) > rest) --i;
    while (i + 1 < s.units && s.start(i + 1, tt) <= rest) ++i;
    unit = i;
    unit_at = at - (rest - s.start(i, tt));
  }
  __device__ __forceinline__ ChunkPiece describe(const ChunkArgs& a) const {
    const int T = a.tile_tokens, tt = 2 * T;
    ChunkPiece p;
    p.b = b;
    p.kvh = kvh;
    p.row0 = s.o0 + unit * tt;
    p.tokens = min(tt, s.n - unit * tt);
    p.first = s.ctx - s.n + unit * tt;
    p.ctx = s.ctx;
    p.kt[0] = (max(p.first + min(p.tokens, T), 0) + kChunkKeys - 1) / kChunkKeys;
    p.kt[1] = p.tokens > T ? (max(p.first + p.tokens, 0) + kChunkKeys - 1) / kChunkKeys : 0;
    return p;
  }
  // The key tile at an offset of the line into the unit.
  __device__ __forceinline__ static int tile_at(int64_t offset, int64_t cost, int tiles) {
    return offset >= cost ? tiles : static_cast<int>(min(offset / kChunkKeys, static_cast<int64_t>(tiles)));
  }
  __device__ __forceinline__ void step(const ChunkArgs& a, int64_t unit_cost) {
    unit_at += unit_cost;
    if (++unit < s.units) return;
    unit = 0;
    if (++kvh < a.num_kv_heads) return;
    kvh = 0;
    while (++b < a.num_seqs) {
      s = chunk_seq(a, b, false, s.whole);
      if (s.n > 0) return;
    }
  }
  // The next piece of this CTA that has something to do.
  __device__ __forceinline__ bool next(const ChunkArgs& a, int cta, ChunkPiece& p) {
    const int tt = 2 * a.tile_tokens;
    while (at < stop && b < a.num_seqs) {
      p = describe(a);
      const int64_t c = cost(tt), from = at - unit_at, to = min(stop - unit_at, c);
      const int tiles = p.tiles();
      p.t0 = tile_at(from, c, tiles);
      p.t1 = tile_at(to, c, tiles);
      p.slot = p.t0 == 0 && p.t1 == tiles ? -1 : p.t0 == 0 ? 2 * cta + 1 : 2 * cta;
      at = unit_at + to;
      if (to == c) step(a, c);
      if (p.t0 < p.t1 || (tiles == 0 && from == 0)) return true;
    }
    return false;
  }
};

// CTA c's part of a line of `total` for `parts` CTAs: [line_cut(c), line_cut(c + 1)).
__device__ __forceinline__ int64_t line_cut(int64_t total, int parts, int c) {
  if (total >> 32 == 0) {  // (a 64-bit quotient is some hundred instructions)
    const uint32_t t = static_cast<uint32_t>(total), p = static_cast<uint32_t>(parts);
    return static_cast<int64_t>(t / p) * c + t % p * c / p;
  }
  return total / parts * c + total % parts * c / parts;
}

// By all threads of a CTA: the length of the line, and what lies before each
// thread's run of sequences (in scratch, one int64 per warp).  Then `find` gives
// the sequence at a place of the line.
struct ChunkLine {
  int64_t total;
  int parts;
  int64_t mine;    // line before this thread's sequences
  int b0, b1;
  bool whole;      // the line counts units

  __device__ __forceinline__ void measure(const ChunkArgs& a, int64_t* scratch, bool flag) {
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.num_seqs + nt - 1) / nt;
    b0 = min(tid * per, a.num_seqs);
    b1 = min(b0 + per, a.num_seqs);
    whole = a.whole_units == 2;
    if (a.whole_units == 1) {
      bool far = false;
      for (int b = b0; b < b1; ++b) far |= __ldg(a.context_lens + b) > kWholeKeys;
      whole = !__syncthreads_or(far);
    }
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += chunk_seq(a, b, flag, whole).line * a.num_kv_heads;
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) scratch[warp] = scan;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < nt / 32; ++w) {
      const int64_t v = scratch[w];
      if (w < warp) before += v;
      total += v;
    }
    mine = before + scan - sum;
    static_assert((kLeastKeys & (kLeastKeys - 1)) == 0, "a shift");
    const int64_t most = whole ? total : total / kLeastKeys;
    parts = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(a.grid), most)));
  }
  // The thread whose sequences hold place x of the line stores (sequence, rest).
  __device__ __forceinline__ void find(const ChunkArgs& a, int64_t x, int64_t* found) const {
    if (x < mine) return;
    int64_t at = mine;
    for (int b = b0; b < b1; ++b) {
      const int64_t l = chunk_seq(a, b, false, whole).line * a.num_kv_heads;
      if (x < at + l) {
        if (x >= at) {
          found[0] = b;
          found[1] = x - at;
        }
        return;
      }
      at += l;
    }
  }
};

// ------------------------------------------------------------------ small pieces

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (x, y) = (x, y) * k + (c, c), each rounded once.
__device__ __forceinline__ void scale2(float& x, float& y, float k, float c) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 w, {%3, %3};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(k), "f"(c));
}
__device__ __forceinline__ void sum2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 u, u, v;\n\t"
      "mov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// 1 / l of a row with reference m (a NaN stays one).
__device__ __forceinline__ float sum_inverse(float m, float l) {
  return l != 0.f ? 1.0f / l : m == kLeastRef ? __int_as_float(0x7fffffff) : 0.f;
}

// 3-D tiled TMA load (dims, heads, tokens) of a box of queries.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A block of a pool, as (64 dims, 8 tokens, D / 64, groups of 8 tokens): a box of two
// groups.  Without a hint for L2, where the CTAs of a (sequence, KV head) find each
// other's tiles.
__device__ __forceinline__ void tma_load_block(uint32_t dst, const CUtensorMap* map, int32_t group, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar)
      : "memory");
}

// First group of 8 tokens of (block, KV head); a block outside the pool reads as zeros.
__device__ __forceinline__ int chunk_pool_group(const ChunkArgs& a, int phys, int kvh) {
  if (phys < 0 || phys >= a.num_blocks) {
    flag_error(kErrBlockId);
    return -2;
  }
  return (phys * a.num_kv_heads + kvh) * 2;
}

// Whether one of a word's two values is infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  constexpr uint32_t kExp = MmaKind<T>::kBf16 ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = MmaKind<T>::kBf16 ? 0x00800080u : 0x04000400u;
  return ((w & kExp) + kOne) & 0x80008000u;
}

// The tile's P V of one row, by its thread: P (packed T) lies in TMEM at p, V in
// shared memory, and only the row's first `vis` keys count.  For tiles with a value
// that is not finite: out of line, and slow.
template <typename T, int D>
__device__ __noinline__ void chunk_row_product(uint32_t p, uint32_t o, const uint8_t* v, int vis, bool fresh) {
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    uint32_t acc[32];
    if (fresh) {
#pragma unroll
      for (int k = 0; k < 32; ++k) acc[k] = 0;
    } else {
      tc::tmem_ld32(o + d, acc);
      tc::tmem_wait_ld();
    }
#pragma unroll 1
    for (int t0 = 0; t0 < kChunkKeys; t0 += 64) {
      uint32_t pk[32];
      __syncwarp();  // (rows of other lengths: the lanes have parted below)
      tc::tmem_ld32(p + t0 / 2, pk);
      tc::tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < 64; ++t) {
        if (t0 + t >= vis) continue;
        const float2 w2 = unpack2<T>(pk[t >> 1]);
        const float w = t & 1 ? w2.y : w2.x;
        const uint8_t* row = v + ((t0 + t) >> 3) * ChunkShape<D>::kGroup + (d >> 6) * ChunkShape<D>::kAtom + (t & 7) * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(row + ((((d & 63) >> 3) + c) ^ ((t0 + t) & 7)) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(word_of(x, i));
            const int k = 8 * c + 2 * i;
            acc[k] = __float_as_uint(fmaf(w, f.x, __uint_as_float(acc[k])));
            acc[k + 1] = __float_as_uint(fmaf(w, f.y, __uint_as_float(acc[k + 1])));
          }
        }
      }
    }
    __syncwarp();
    tc::tmem_st32(o + d, acc);
  }
  tc::tmem_wait_st();
}

// ------------------------------------------------------------------ main kernel

template <typename T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const ChunkArgs a) {
  using Shape = ChunkShape<D>;
  constexpr int NS = Shape::kSlots;
  constexpr bool kBf16 = MmaKind<T>::kBf16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[NS], ready[kChunkSteps], done[kChunkSteps];
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], p_early[2], p_full[2], o_full[2], turn[2], mma_fin[2];
  __shared__ int64_t s_found[2];
  __shared__ __align__(8) uint64_t piece_full[kChunkPieces], piece_empty[kChunkPieces];
  __shared__ ChunkPiece s_piece[kChunkPieces];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_slow[kChunkSteps];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_smem = base;
  uint8_t* ring = base + 2 * Shape::kTileBytes;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
    }
    for (int s = 0; s < kChunkSteps; ++s) {
      mbar_init(smem_u32(&ready[s]), 1);
      mbar_init(smem_u32(&done[s]), 2);
    }
    for (int s = 0; s < kChunkPieces; ++s) {
      mbar_init(smem_u32(&piece_full[s]), 1);
      mbar_init(smem_u32(&piece_empty[s]), 2 + 1 + 8);  // the MMA warps, the V warp, the softmax warps
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_empty), 2);
    for (int q = 0; q < 2; ++q) {
      mbar_init(smem_u32(&s_full[q]), 1);
      mbar_init(smem_u32(&p_early[q]), 4);
      mbar_init(smem_u32(&p_full[q]), 4);
      mbar_init(smem_u32(&o_full[q]), 1);
      mbar_init(smem_u32(&turn[q]), 1);
      mbar_init(smem_u32(&mma_fin[q]), 1);
    }
    s_abort = 0;
    s_found[0] = -1;
    fence_mbar_init();
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  if (warp == 9) {
    tc::tmem_alloc(smem_u32(&s_tmem), Shape::kTmemCols);
    tc::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = blockIdx.x;
  int64_t at = 0, stop = 0;  // this CTA's part of the line
  bool whole;
  {
    ChunkLine line;
    line.measure(a, reinterpret_cast<int64_t*>(ring), cta == 0);  // (the ring is not in use yet)
    if (cta < line.parts) {
      at = line_cut(line.total, line.parts, cta);
      stop = line_cut(line.total, line.parts, cta + 1);
    }
    if (at < stop) line.find(a, at, s_found);
    whole = line.whole;
  }
  tc::fence_before_sync();
  fence_proxy_async_smem();  // the scratch in the ring, before its first tile
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = s_tmem;
  volatile int* abort_flag = &s_abort;
  // The other warps' next piece: where the TMA warp has put it, or null.  The slot
  // is theirs until they release it.
  uint32_t pieces = 0;
  auto take = [&](bool whole_warp) -> const ChunkPiece* {
    const uint32_t slot = pieces % kChunkPieces;
    bool ok = mbar_wait(smem_u32(&piece_full[slot]), (pieces / kChunkPieces) & 1) && !*abort_flag;
    if (whole_warp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      *abort_flag = 1;
      return nullptr;
    }
    ++pieces;
    return s_piece[slot].b >= 0 ? &s_piece[slot] : nullptr;
  };
  auto release = [&]() { mbar_arrive(smem_u32(&piece_empty[(pieces - 1) % kChunkPieces])); };

  // The launch's 384 x 168 registers are divided anew: 256 x 208 + 128 x 88.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ------------------------------------------------------------ TMA
      ChunkWalk walk;
      walk.at = at;
      walk.stop = stop;
      walk.b = a.num_seqs;
      if (at < stop) walk.locate(a, static_cast<int>(s_found[0]), s_found[1], whole);
      uint32_t it = 0;      // tiles issued
      uint32_t steps = 0;   // of the MMA warps before this piece
      uint32_t seen_done = 0, slot_step = 0;  // lane s: the step of the tile in slot s
      int loads = 0;        // of queries
      bool ok = true;
      bool first = true;
      for (bool last = false; ok && !last;) {
        ChunkPiece p;
        last = !walk.next(a, cta, p);
        if (last) p.b = -1;
        if (first && lane == 0) {
          ChunkCut c = {};
          if (!last && p.t0 > 0) c = {1, p.t1 < p.tiles(), p.row0, p.tokens, p.kvh};
          a.cuts[cta] = c;
        }
        first = false;
        const uint32_t slot = pieces % kChunkPieces;
        if (pieces >= kChunkPieces) ok = mbar_wait(smem_u32(&piece_empty[slot]), (pieces / kChunkPieces - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (lane == 0) {
          s_piece[slot] = p;
          mbar_arrive(smem_u32(&piece_full[slot]));
        }
        __syncwarp();
        ++pieces;
        if (last || p.t0 == p.t1) continue;
        // Queries, once every S of the piece before is done.
        if (loads > 0) ok = mbar_wait(smem_u32(&q_empty), (loads - 1) & 1);
        ++loads;
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (lane == 0) {
          const int tiles = p.t0 < p.kt[1] ? 2 : 1;
          mbar_arrive_expect_tx(smem_u32(&q_full), tiles * (D / 64) * a.tile_tokens * a.group * 128);
          for (int q = 0; q < tiles; ++q)
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
              tma_load_3d(smem_u32(q_smem) + q * Shape::kTileBytes + d * Shape::kQHalf, &tmap_q, 64 * d,
                          p.kvh * a.group, p.row0 + q * a.tile_tokens, smem_u32(&q_full));
        }
        const int32_t* table = a.block_tables + static_cast<int64_t>(p.b) * a.max_blocks;
        const int nblk = (p.ctx + kBlockSize - 1) / kBlockSize;
        int win = -32, row = 0;
        for (int t = p.t0; t < p.t1 && ok; ++t) {
          const int blk = t * (kChunkKeys / kBlockSize);
          if (blk >= win + 32) {
            win = blk;
            row = win + lane < nblk ? chunk_pool_group(a, __ldg(table + win + lane), p.kvh) : 0;
          }
          const int mine = __shfl_sync(0xffffffffu, row, blk - win + (lane & 7));
          const int here = min(kChunkKeys / kBlockSize, nblk - blk);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {  // K, then V
            const int slot = it % NS;
            // The slot's last tile is done with when its step is (all before it too).
            const uint32_t last_step = __shfl_sync(0xffffffffu, slot_step, slot);
            if (it >= NS)
              for (; ok && seen_done <= last_step; ++seen_done)
                ok = mbar_wait(smem_u32(&done[seen_done % kChunkSteps]), (seen_done / kChunkSteps) & 1);
            if (lane == slot) slot_step = steps + (t - p.t0) + kv;  // V of a tile goes with K of the next
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            const uint32_t bar = smem_u32(&kv_full[slot]);
            const uint32_t dst = smem_u32(ring) + slot * Shape::kTileBytes;
            if (lane == 0) mbar_arrive_expect_tx(bar, here * kBlockSize * D * 2);
            __syncwarp();
            if (lane < here) tma_load_block(dst + lane * 2 * Shape::kGroup, kv ? &tmap_v : &tmap_k, mine, bar);
          }
        }
        steps += p.t1 - p.t0 + 1;
      }
      if (!ok) {
        *abort_flag = 1;
        // No copy may still be landing in shared memory at exit.
        if (loads > 0) mbar_wait(smem_u32(&q_full), (loads - 1) & 1);
        for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait(smem_u32(&kv_full[i % NS]), (i / NS) & 1);
      }
    } else if (warp < 11) {
      // ------------------------------------------------------------ MMA of one tile
      if (lane == 0) {
        const int q = warp - 9;
        const uint32_t idesc_s = tc::idesc_f16(kBf16, 128, kChunkKeys, false) | (a.negate ? 1u << 13 : 0u);
        constexpr uint32_t idesc_o = tc::idesc_f16(kBf16, 128, D, true);
        const uint32_t s_col = tbase + Shape::kSCol + 128 * q, o_col = tbase + Shape::kOCol + D * q;
        const uint64_t q_desc = tc::smem_desc_sw128(smem_u32(q_smem) + q * Shape::kTileBytes, 16, 1024);
        uint32_t slot = 0, step = 0;  // the next K or V tile's, as the TMA warp counts them; the next step
        uint32_t np = 0, loads = 0;
        bool ok = true;
        auto next_slot = [&]() {
          const uint32_t x = slot;
          slot = slot + 1 == NS ? 0 : slot + 1;
          return x;
        };
        // A and B issue in turn: left to themselves they fall into phase, both tiles'
        // products queued at once and then both softmaxes (461 us against 361).
        uint32_t turns = 0;
        auto my_turn = [&]() {
          const uint32_t n = turns++;
          return q == 0 ? n == 0 || mbar_wait(smem_u32(&turn[0]), (n - 1) & 1) : mbar_wait(smem_u32(&turn[1]), n & 1);
        };
        auto pass_on = [&]() { mbar_arrive(smem_u32(&turn[q ^ 1])); };
        while (const ChunkPiece* next = take(false)) {
          const int t0 = next->t0, t1 = next->t1, kt = next->kt[q];
          const int masked_from = max(next->first + 1, 0) / kChunkKeys;  // first tile that not every row sees whole
          release();
          if (t0 == t1) continue;
          ok = mbar_wait(smem_u32(&q_full), loads++ & 1);
          // A step issues P V of tile t and S of tile t + 1 (the first one only S).
          for (int t = t0 - 1; t < t1 && ok; ++t, ++step) {
            const bool pv = t >= t0 && t < kt, sc = t + 1 < t1 && t + 1 < kt;
            ok = mbar_wait(smem_u32(&ready[step % kChunkSteps]), (step / kChunkSteps) & 1);
            const bool slow = t >= masked_from && *reinterpret_cast<volatile int*>(&s_slow[step % kChunkSteps]) != 0;
            const uint32_t vslot = t >= t0 ? next_slot() : 0, kslot = t + 1 < t1 ? next_slot() : 0;
            if (pv) ok = ok && mbar_wait(smem_u32(&p_early[q]), np & 1);
            ok = ok && my_turn();
            if (!ok) break;
            tc::fence_after_sync();
            if (pv) {
              const uint64_t v_desc =
                  tc::smem_desc_sw128(smem_u32(ring) + vslot * Shape::kTileBytes, Shape::kAtom, Shape::kGroup);
              auto product = [&](int k) {
                tc::mma_ts(o_col, s_col + 8 * k, v_desc + (k * 2 * Shape::kGroup >> 4), idesc_o, t > t0 || k > 0 ? 1u : 0u);
              };
              if (!slow) {
#pragma unroll
                for (int k = 0; k < 2 * kEarly; ++k) product(k);
              }
              ok = mbar_wait(smem_u32(&p_full[q]), np++ & 1);
              if (!ok) break;
              tc::fence_after_sync();
              if (!slow) {
#pragma unroll
                for (int k = 2 * kEarly; k < kChunkKeys / 16; ++k) product(k);
              }
            }
            if (sc) {
              const uint64_t k_desc = tc::smem_desc_sw128(smem_u32(ring) + kslot * Shape::kTileBytes, 16, Shape::kGroup);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tc::mma_ss(s_col, q_desc + (((k >> 2) * Shape::kQHalf + (k & 3) * 32) >> 4),
                           k_desc + (((k >> 2) * Shape::kAtom + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
              tc::mma_commit(smem_u32(&s_full[q]));
            }
            pass_on();
            if (pv && t + 1 == min(t1, kt)) tc::mma_commit(smem_u32(&o_full[q]));
            // The step's tiles are done with once what was issued is.
            if (pv || sc)
              tc::mma_commit(smem_u32(&done[step % kChunkSteps]));
            else
              mbar_arrive(smem_u32(&done[step % kChunkSteps]));
            if (t + 2 == t1) {
              if (t0 < kt)
                tc::mma_commit(smem_u32(&q_empty));
              else
                mbar_arrive(smem_u32(&q_empty));
            }
          }
          if (!ok || *abort_flag) break;
        }
        if (!ok) *abort_flag = 1;
        // No MMA may still be running when the CTA frees its TMEM.
        tc::mma_commit(smem_u32(&mma_fin[q]));
        mbar_wait(smem_u32(&mma_fin[q]), 0);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ V of masked tiles
      uint32_t slot = 0, phase = 0, step = 0;
      bool ok = true;
      auto landed = [&]() {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&kv_full[slot]), phase) && !*abort_flag);
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      };
      while (const ChunkPiece* next = take(true)) {
        const int first = next->first, t0 = next->t0, t1 = next->t1, ctx = next->ctx;
        __syncwarp();
        if (lane == 0) release();
        if (t0 == t1) continue;
        const int seen = max(first + 1, 0);  // keys that every row sees
        for (int t = t0 - 1; t < t1; ++t, ++step) {  // V of tile t, K of tile t + 1
          bool slow = false;
          uint8_t* v = ring + slot * Shape::kTileBytes;
          if (t >= t0) landed();
          if (!ok) break;
          if (t >= t0 && (t + 1) * kChunkKeys > seen) {
            const int from = max(seen - t * kChunkKeys, 0), valid = min(kChunkKeys, ctx - t * kChunkKeys);
            uint32_t bad = 0;
            // 16 bytes a lane, D / 8 lanes a row.
#pragma unroll 4
            for (int x = from * (D / 8) + lane; x < valid * (D / 8); x += 32) {
              const int r = x / (D / 8), c = x % (D / 8);
              const uint4 w = *reinterpret_cast<const uint4*>(v + (r >> 3) * Shape::kGroup + (c >> 3) * Shape::kAtom + (r & 7) * 128 + (c & 7) * 16);
              bad |= not_finite2<T>(w.x) | not_finite2<T>(w.y) | not_finite2<T>(w.z) | not_finite2<T>(w.w);
            }
            for (int x = valid * (D / 8) + lane; x < kChunkKeys * (D / 8); x += 32) {
              const int r = x / (D / 8), c = x % (D / 8);
              *reinterpret_cast<uint4*>(v + (r >> 3) * Shape::kGroup + (c >> 3) * Shape::kAtom + (r & 7) * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            slow = __any_sync(0xffffffffu, bad != 0);
          }
          if (t + 1 < t1) landed();
          if (!ok) break;
          __syncwarp();
          if (lane == 0) {
            s_slow[step % kChunkSteps] = slow;
            mbar_arrive(smem_u32(&ready[step % kChunkSteps]));
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax
    const int q = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tbase + lane_base + Shape::kSCol + 128 * q;
    const uint32_t o_addr = tbase + lane_base + Shape::kOCol + D * q;
    const int tok = q * a.tile_tokens + r / a.group;  // token of the unit
    const bool whole_row = r < a.tile_tokens * a.group;
    const float c2 = a.c2;
    uint32_t ns = 0, no = 0;
    uint32_t it = 0, step = 0;  // K and V tiles, and steps, before this piece
    bool ok = true;
    while (const ChunkPiece* next = take(true)) {
      const ChunkPiece& p = *next;
      const bool valid_row = whole_row && tok < p.tokens;
      // Last position the row attends to.  Rows without a token may come out as anything;
      // a warp of them leaves its weights alone.
      const int limit = valid_row ? p.first + tok : INT_MAX / 2;
      const bool idle = !__any_sync(0xffffffffu, valid_row);
      const int seen = max(p.first + 1, 0);
      const int t0 = p.t0, t1 = p.t1, kt = p.kt[q];
      float m = limit < 0 ? kNoKeysRef : kLeastRef, l = 0.f;
      for (int t = t0; t < t1 && ok; ++t) {
        if (t >= kt) break;  // the other tile's
        ok = mbar_wait(smem_u32(&s_full[q]), ns++ & 1);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (idle) {
          if (lane == 0) {
            mbar_arrive(smem_u32(&p_early[q]));
            mbar_arrive(smem_u32(&p_full[q]));
          }
          __syncwarp();
          continue;
        }
        tc::fence_after_sync();
        uint32_t x[4][32];  // scores as their bits
#pragma unroll
        for (int j = 0; j < 4; ++j) tc::tmem_ld32(s_addr + 32 * j, x[j]);
        tc::tmem_wait_ld();
        const int vis = limit + 1 - t * kChunkKeys;
        if (__any_sync(0xffffffffu, vis < kChunkKeys)) {
#pragma unroll
          for (int k = 0; k < 128; ++k) x[k >> 5][k & 31] = k < vis ? x[k >> 5][k & 31] : 0xff800000u;
        }
        float l0, l1, l2, l3;
        auto weights = [&](int j, float nr) {  // of 32 keys, into TMEM
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __uint_as_float(x[j][2 * k + i]);
            scale2(y[0], y[1], c2, nr);
            scale2(y[2], y[3], c2, nr);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = exp2_approx(y[i]);
            sum2(l0, l1, y[0], y[1]);
            sum2(l2, l3, y[2], y[3]);
            // Weights rounded to T: 2^-8 (bf16) or 2^-11 (fp16) of each at most, beside an
            // output rounded to T; two terms would double the product's work.
            pk[k] = pack2<T>(y[0], y[1]);
            pk[k + 1] = pack2<T>(y[2], y[3]);
          }
          tc::tmem_st16(s_addr + 16 * j, pk);
        };
        // The first weights are made with the reference there is while the maxima are
        // found, and made again if it has to move: when a score passes it by 2^8.
        l0 = l1 = l2 = l3 = 0.f;
        float nr = -m;
        if (t > t0) {
#pragma unroll
          for (int j = 0; j < kEarly; ++j) weights(j, nr);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = fmaxf(mx[i], fmaxf(__uint_as_float(x[k >> 5][(k & 31) + 2 * i]), __uint_as_float(x[k >> 5][(k & 31) + 2 * i + 1])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        const bool up = top > m + 8.f;
        if (t == t0 || __any_sync(0xffffffffu, up)) {
          const float al = up ? exp2_approx(m - top) : 1.f;
          if (t > t0) {
            // P V of the tiles before is done: S of this tile was issued after it.
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              uint32_t o[16];
              tc::tmem_ld16(o_addr + 16 * j, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
              tc::tmem_st16(o_addr + 16 * j, o);
            }
          }
          l *= al;
          if (up) m = top;
          nr = -m;
          l0 = l1 = l2 = l3 = 0.f;
#pragma unroll
          for (int j = 0; j < kEarly; ++j) weights(j, nr);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_early[q]));  // their part of P V may begin
#pragma unroll
        for (int j = kEarly; j < 4; ++j) weights(j, nr);
        l += (l0 + l1) + (l2 + l3);
        tc::tmem_wait_st();
        if ((t + 1) * kChunkKeys > seen) {
          const uint32_t sv = step + (t - t0) + 1, iv = it + 2 * (t - t0) + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ready[sv % kChunkSteps]), (sv / kChunkSteps) & 1));
          if (!ok) break;
          if (*reinterpret_cast<volatile int*>(&s_slow[sv % kChunkSteps]) != 0)
            chunk_row_product<T, D>(s_addr, o_addr, ring + (iv % NS) * Shape::kTileBytes, vis, t == t0);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[q]));
      }
      if (!ok) break;
      it += 2 * (t1 - t0);
      if (t0 < t1) step += t1 - t0 + 1;
      const bool any = t0 < kt;
      if (any) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&o_full[q]), no++ & 1));
        if (!ok) break;
        tc::fence_after_sync();
      }
      const int64_t orow = (static_cast<int64_t>(p.row0) + tok) * a.num_q_heads + p.kvh * a.group + r % a.group;
      const float inv = sum_inverse(m, l);
      float* part = p.slot >= 0 ? a.part + p.slot * Shape::kPart : nullptr;
      // A lane holds a row, and 32 stores of 16 bytes to 32 rows are 32 accesses.  So the
      // output goes through exchanges within four lanes, after which each has the same
      // 16 bytes of every 64 of their four rows; partial results lie as they are held.
      int64_t rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xffffffffu, valid_row ? orow : -1, (lane & ~3) + i);
#pragma unroll 1
      for (int j = 0; j < (idle ? 0 : D / 32); ++j) {
        uint32_t o[32];
        if (any) {
          tc::tmem_ld32(o_addr + 32 * j, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (part) {
          uint4* dst = reinterpret_cast<uint4*>(part) + (8 * j) * kChunkRows + q * 128 + r;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k * kChunkRows] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = pack2<T>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          // v[4 c + w]: word w of the row's 16 bytes c; then of row c of the four, 16 bytes (lane % 4).
#pragma unroll
          for (int h = 1; h <= 2; h *= 2) {
            const bool odd = lane & h;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c & h) continue;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t give = odd ? v[4 * c + w] : v[4 * (c + h) + w];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, h);
                if (odd)
                  v[4 * c + w] = got;
                else
                  v[4 * (c + h) + w] = got;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (rows[c] >= 0)
              reinterpret_cast<uint4*>(static_cast<T*>(a.out) + rows[c] * D + 32 * j)[lane & 3] =
                  make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        }
        __syncwarp();
      }
      if (part && valid_row) {
        part[kChunkRows * D + q * 128 + r] = m;
        part[kChunkRows * (D + 1) + q * 128 + r] = l;
      }
      tc::fence_before_sync();  // O has been read: the next piece's first product, after this row's next P, may write it
      __syncwarp();
      if (lane == 0) release();
    }
    if (!ok) *abort_flag = 1;
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, Shape::kTmemCols);
  }
}

// ------------------------------------------------------------------ merge

constexpr int kChunkMergeThreads = 256;
constexpr int kChunkMergeRows = 32;

// CTA (c, y) joins the pieces of the unit inside which CTA c's part begins, if that is
// the unit's first cut, for 32 of its rows, four a warp: the last piece of CTA c - 1,
// the first of CTA c, and those of the CTAs after it as long as their whole part lay in
// the unit.  40 MB of partial results at most; 9 to 12 us, a chain of cut, pieces, row.
// (Finding the cuts from the lengths again instead of reading them: 34 us.)
template <typename T, int D>
__global__ void __launch_bounds__(kChunkMergeThreads) merge_chunk_kernel(const ChunkArgs a) {
  using Shape = ChunkShape<D>;
  constexpr int kPer = D / 32, kRows = kChunkMergeRows / (kChunkMergeThreads / 32);
  static_assert(kRows == 4, "four rows a warp");
  const int c = blockIdx.x + 1;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto cut_of = [&](int x) {
    const int4* p = reinterpret_cast<const int4*>(a.cuts + x);
    const int4 u = __ldcg(p), v = __ldcg(p + 1);
    return ChunkCut{u.x, u.y, u.z, u.w, v.x};
  };
  const ChunkCut here = cut_of(c), prev = cut_of(c - 1);
  if (!here.cut || (prev.cut && prev.open)) return;
  const int rows = here.tokens * a.group, half = a.tile_tokens * a.group;  // half: rows of tile A
  const int r0 = blockIdx.y * kChunkMergeRows + (threadIdx.x >> 5) * kRows;  // rows of the unit, tokens packed
  if (r0 >= rows) return;
  // Lane: row r0 + lane % 4, dims 4 (lane / 4) + 32 k.
  const int rr = r0 + (lane & 3);
  const int pr = min(rr, rows - 1) < half ? min(rr, rows - 1) : 128 + min(rr, rows - 1) - half;  // its place in a partial result
  float M = kLeastRef, L = 0.f;
  float4 o[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  int slot = 2 * c - 1;
  bool open = here.open;
  for (int x = c;;) {
    const float* src = a.part + slot * Shape::kPart;
    const float m = __ldcg(src + kChunkRows * D + pr), l = __ldcg(src + kChunkRows * (D + 1) + pr);
    float4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(src) + ((lane >> 2) + 8 * k) * kChunkRows + pr);
    // (A piece without any weight, kLeastRef, counts 0; its O is 0, or NaN by a V that is not
    // finite.)
    const float top = fmaxf(M, m), wo = exp2f(M - top), wn = exp2f(m - top);
    L = L * wo + l * wn;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      o[k] = make_float4(o[k].x * wo + v[k].x * wn, o[k].y * wo + v[k].y * wn, o[k].z * wo + v[k].z * wn,
                         o[k].w * wo + v[k].w * wn);
    M = top;
    if (slot & 1) {
      slot = 2 * c;  // after the first piece, CTA c's
    } else {
      if (!open || x + 1 >= a.grid) break;
      slot = 2 * ++x;
      open = cut_of(x).open;
    }
  }
  if (rr >= rows) return;
  const float inv = sum_inverse(M, L);
  const int64_t orow = (static_cast<int64_t>(here.row0) + rr / a.group) * a.num_q_heads + here.kvh * a.group + rr % a.group;
  T* dst = static_cast<T*>(a.out) + orow * D + 4 * (lane >> 2);
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    *reinterpret_cast<uint2*>(dst + 32 * k) =
        make_uint2(pack2<T>(o[k].x * inv, o[k].y * inv), pack2<T>(o[k].z * inv, o[k].w * inv));
}

}  // namespace pkv
