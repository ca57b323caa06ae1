// Decode attention over a 4-bit pool (sm_103a): one persistent CTA per SM, the
// (sequence, KV head, block) space in equal shares, one per warp, and the early
// reads before the grid wait of decode_persistent_kernel; then a merge of the
// units that shares cut (merge_int4_kernel).
//
// A token is a quarter of a bf16 pool's bytes, so at the same bandwidth a warp
// has a quarter of the instructions per token.  What the kernel does about it:
//   * a stage is up to four blocks of one unit, described when a window of 32
//     table entries is read (all lanes at once);
//   * codes are multiplied without a conversion (WarpAttnInt4);
//   * the softmax step covers a stage and mostly needs no cross-lane work.
#pragma once

#include "int4_cache.cuh"
#include "paged_kv_kernels.cuh"

namespace pkv {

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// d += A * B and d = A * B in fp16 with fp32 accumulation.  Not volatile: the
// compiler may interleave the independent chains.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ===================================================================== warp math

// One warp's attention state for one (sequence, KV head) unit over 4-bit tiles.
//
// Codes go to the tensor cores without a conversion: a code masked out of its
// word in place, c or 16 c in the low bits of a 16-bit half, is the float16
// subnormal c * 2^-24 or c * 2^-20, which mma.sync multiplies exactly.  Eight
// codes cost one shift and four ANDs.
//   scores:  q . K_t = s_t (q . c_t) + m_t sum(q)            (float32, per token)
//   output:  sum_t p_t V_t = sum_t P_t c_t + sum_t p_t m_t,  P_t = p_t s_t
// P is rounded to float16, and the rounding must act on c - 7.5 and not on c,
// whose common part is several times the value: with a = sum of the rounded P
// (one more mma, against ones),
//   sum P_t c_t + sum p_t m_t = [sum P_t c_t - 7.5 a] + sum p_t (m_t + 7.5 s_t).
// The bracket is formed every kFlushBlocks blocks (flush), which also keeps
// the accumulators at the output's size: an accumulator that carried 7.5 a
// over a long context would lose the output's low bits to it.
//
// The softmax reference M (p_t = 2^(x_t - M)) is not the maximum but what keeps
// P within float16 and its largest value well inside: M moves so that the largest
// product p_t s_t met, and not the largest p_t or s_t, lies at 2^kTarget when it
// moves and below 2^kTop always.  A row's rounding error is then 2^-11 of its own
// P, or 2^-25 where the largest is at least 1, whatever the scales of rows that
// carry no weight.  (A scale of 0 counts as 2^-24, float16's smallest, so that p
// stays below 2^38.  Scales count by their exponent, which makes the heaviest
// row's p a power of two: a context of one token returns its row.)
// Most steps need no look at the products: scores up to `limit` above M and
// scales up to a cap C, limit = kTop - log2 C, cannot exceed 2^kTop; one vote, no
// shuffles, no rescaling.  C is 2^kScaleSlack times the largest scale of the last
// step that failed this; it decides only which steps are looked at.
//
// Lane (gid = lane/4, c = lane%4): scores of tokens gid, gid + 8 and heads 2c,
// 2c + 1 as in WarpAttn; O^T entries of dims [G gid, G gid + G), G = D/8.
template <typename T, int D>
struct WarpAttnInt4 {
  using Tile = Int4Tile<D>;
  static constexpr int kWords = D / 32;  // 32-bit words of codes per lane and row
  static constexpr int kFlushBlocks = 64;
  static constexpr float kTop = 14.f;    // log2; float16's largest is 65504
  static constexpr float kTarget = 0.f;  // log2: room below kTop for later scores (8) and scales (6)
  static constexpr int kScaleSlack = 6;  // log2, for later scales
  static constexpr float kTiny = 5.9604644775390625e-8f;  // 2^-24
  uint32_t qf[4 * kWords];
  float acc[D / 16][4];
  float ones[4];         // sum of rounded P since the last flush (heads 2c, 2c + 1; twice)
  float m0, m1, l0, l1;  // softmax reference (log2 units) and sum of p
  float b0, b1;          // sum of p (m + 7.5 s)
  float qs0, qs1;        // scale_log2 * sum(q)
  float cap, limit;      // C, and how far a score may exceed the reference untested; cap < 0 before the first step
  int since_flush;       // blocks

  __device__ __forceinline__ void reset() {
    m0 = m1 = l0 = l1 = b0 = b1 = 0.f;
    cap = -1.f;
    limit = 0.f;
    since_flush = 0;
    ones[0] = ones[1] = ones[2] = ones[3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }

  // Entries [(D/4) c, (D/4) (c + 1)) of query row gid as float16 in the order
  // the masked K words pair them; a bf16 query beyond the float16 range is
  // flagged (kErrQuery), below its normal range (2^-14) it is off by 2^-25 at most.  Word w holds dims d0..d7: registers (d0,d4), (d2,d6)
  // meet the masks of factor 1, (d1,d5), (d3,d7) those of factor 16.
  __device__ __forceinline__ void load_q(const T* q_group, int group, float scale_log2, int lane) {
    const int gid = lane >> 2, c = lane & 3;
    bool big = false;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint4 raw = gid < group ? __ldg(reinterpret_cast<const uint4*>(q_group + gid * D + (D / 4) * c) + w)
                                    : make_uint4(0, 0, 0, 0);
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(word_of(raw, i));
        if constexpr (MmaKind<T>::kBf16) {
          big |= fabsf(f.x) > kF16Max || fabsf(f.y) > kF16Max;
          h[i] = pack2<__half>(f.x, f.y);
          const float2 g = unpack2<__half>(h[i]);
          sum += g.x + g.y;
        } else {
          h[i] = word_of(raw, i);
          sum += f.x + f.y;
        }
      }
      qf[4 * w] = __byte_perm(h[0], h[2], 0x5410);
      qf[4 * w + 1] = __byte_perm(h[1], h[3], 0x5410);
      qf[4 * w + 2] = __byte_perm(h[0], h[2], 0x7632);
      qf[4 * w + 3] = __byte_perm(h[1], h[3], 0x7632);
    }
    if (__any_sync(0xffffffffu, big) && lane == 0) flag_error(kErrQuery);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    qs0 = scale_log2 * __shfl_sync(0xffffffffu, sum, 8 * c);
    qs1 = scale_log2 * __shfl_sync(0xffffffffu, sum, 8 * c + 4);
  }

  __device__ __forceinline__ static void load_words(const uint8_t* p, uint32_t (&w)[kWords]) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }

  static constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kBoth = 0x00ff00ffu;

  // 2^-24 (q . c) of tokens gid (x[.][0..1]) and gid + 8 (x[.][2..3]), heads 2c
  // and 2c + 1, of NB blocks' K tiles (2 * kBytes apart): 2 NB independent mma
  // chains, interleaved.
  template <int NB>
  __device__ __forceinline__ void dots(const uint8_t* ks, int lane, float (&x)[NB][4]) const {
    float t[NB][4];
    uint32_t wa[NB][kWords], wb[NB][kWords];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      load_words(ks + i * 2 * Tile::kBytes + lane * (D / 8), wa[i]);                         // row gid, quarter c
      load_words(ks + i * 2 * Tile::kBytes + Tile::kCodeBytes / 2 + lane * (D / 8), wb[i]);  // row gid + 8
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t a = wa[i][w], b = wb[i][w], a8 = a >> 8, b8 = b >> 8;
        if (w == 0) {
          mma_f16_first(x[i], a & kLow, b & kLow, a8 & kLow, b8 & kLow, qf[0], qf[1]);
          mma_f16_first(t[i], a & kHigh, b & kHigh, a8 & kHigh, b8 & kHigh, qf[2], qf[3]);
        } else {
          mma_f16(x[i], a & kLow, b & kLow, a8 & kLow, b8 & kLow, qf[4 * w], qf[4 * w + 1]);
          mma_f16(t[i], a & kHigh, b & kHigh, a8 & kHigh, b8 & kHigh, qf[4 * w + 2], qf[4 * w + 3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      fma2(x[i][0], x[i][1], t[i][0], t[i][1], 0.0625f, x[i][0], x[i][1]);
      fma2(x[i][2], x[i][3], t[i][2], t[i][3], 0.0625f, x[i][2], x[i][3]);
    }
  }

  // acc += V^T P^T for one tile, times 2^-24: m-tile 2w holds dims 4w (rows gid)
  // and 4w + 2 (rows gid + 8) of the lane's G, m-tile 2w + 1 those plus 16 times
  // dims 4w + 1 and 4w + 3.  A byte with both its codes c + 16 c' is a float16
  // subnormal too, and takes one operation less to cut out than c' alone; the
  // two are told apart at the end (chunk_values).
  __device__ __forceinline__ void pv(const uint8_t* vs, uint32_t p0, uint32_t p1, int lane) {
    uint32_t x[kWords], y[kWords];
    load_words(vs + lane * (D / 8), x);                         // tokens 2c, 2c + 1
    load_words(vs + Tile::kCodeBytes / 2 + lane * (D / 8), y);  // tokens 2c + 8, 2c + 9
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t x8 = __byte_perm(x[w], 0, 0x4341), y8 = __byte_perm(y[w], 0, 0x4341);  // bytes 1 and 3
      mma_f16(acc[2 * w], x[w] & kLow, x8 & kLow, y[w] & kLow, y8 & kLow, p0, p1);
      mma_f16(acc[2 * w + 1], x[w] & kBoth, x8, y[w] & kBoth, y8, p0, p1);
    }
  }

  // Sum over the lanes that share c.
  __device__ __forceinline__ static float sum_gid(float v) {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  __device__ __forceinline__ void flush() {
    const float f0 = ones[0] * (7.5f * kTiny), f1 = ones[1] * (7.5f * kTiny);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float u = i & 1 ? -17.f : -1.f;
      acc[i][0] = fmaf(u, f0, acc[i][0]);
      acc[i][1] = fmaf(u, f1, acc[i][1]);
      acc[i][2] = fmaf(u, f0, acc[i][2]);
      acc[i][3] = fmaf(u, f1, acc[i][3]);
    }
    ones[0] = ones[1] = ones[2] = ones[3] = 0.f;
    since_flush = 0;
  }

  // The references for a step that failed the quick test (or the first): up, so
  // that the largest product lies at 2^kTarget, where it lies above; x (scores
  // less the reference) and what was summed so far follow.
  template <int NB>
  __device__ __forceinline__ void move_reference(float (&x)[NB][4], const float (&sv)[NB][2], float smax) {
    float d0 = -INFINITY, d1 = -INFINITY;  // log2 of the largest products, less 1 at most
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      // log2 of the scales, rounded down: their exponents as the low bits of 2^23's.
      float la = __uint_as_float(__funnelshift_r(__float_as_uint(fmaxf(fabsf(sv[i][0]), kTiny)), 0x4b000000u >> 9, 23));
      float lb = __uint_as_float(__funnelshift_r(__float_as_uint(fmaxf(fabsf(sv[i][1]), kTiny)), 0x4b000000u >> 9, 23));
      add2(la, lb, -(8388608.f + 127.f), -(8388608.f + 127.f));
      float y0 = x[i][0], y1 = x[i][1], y2 = x[i][2], y3 = x[i][3];
      add2(y0, y1, la, la);
      add2(y2, y3, lb, lb);
      d0 = max3(d0, y0, y2);
      d1 = max3(d1, y1, y3);
    }
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      d0 = fmaxf(d0, __shfl_xor_sync(0xffffffffu, d0, o));
      d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, o));
    }
    const bool first = cap < 0.f;  // nothing is summed yet: the references may also go down
    // The bits of floats >= 0 order as they do; the exponent is all that counts.
    const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(smax, kTiny))) >> 23;
    cap = __uint_as_float((e + kScaleSlack) << 23);
    limit = kTop - static_cast<float>(static_cast<int>(e) + kScaleSlack - 127);
    d0 -= kTarget;
    d1 -= kTarget;
    if (!first) {
      d0 = fmaxf(d0, 0.f);
      d1 = fmaxf(d1, 0.f);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      add2(x[i][0], x[i][1], -d0, -d1);
      add2(x[i][2], x[i][3], -d0, -d1);
    }
    m0 += d0;
    m1 += d1;
    if (!first) {
      const float al0 = exp2_approx(-d0), al1 = exp2_approx(-d1);
      l0 *= al0;
      l1 *= al1;
      b0 *= al0;
      b1 *= al1;
      ones[0] *= al0;
      ones[1] *= al1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        acc[i][0] *= al0;
        acc[i][1] *= al1;
        acc[i][2] *= al0;
        acc[i][3] *= al1;
      }
    }
  }

  // One softmax step over NB consecutive blocks of one unit, whose (K tile, V
  // tile) pairs lie back to back at `stage`.  MASK: only the first `valid` (1..16
  // NB) tokens belong to the context; pairs and codes of the slots behind them
  // may hold anything, their scores and scales are replaced.
  template <int NB, bool MASK>
  __device__ __forceinline__ void step(const uint8_t* stage, int valid, float scale_log2, int lane) {
    const int gid = lane >> 2;
    const float k_mul = scale_log2 * 16777216.f;  // 2^24
    float x[NB][4], sv[NB][2], mv[NB][2];         // scores less the reference; V's scales and minima
    float d0 = -INFINITY, d1 = -INFINITY, smax = 0.f;
    if constexpr (NB % 2 == 0) {
#pragma unroll
      for (int i = 0; i < NB; i += 2) dots<2>(stage + i * 2 * Tile::kBytes, lane, reinterpret_cast<float(&)[2][4]>(x[i]));
    } else {
      dots<NB>(stage, lane, x);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint8_t* ks = stage + i * 2 * Tile::kBytes;
      const uint32_t* km = reinterpret_cast<const uint32_t*>(ks + Tile::kCodeBytes) + gid;
      const uint32_t* vm = reinterpret_cast<const uint32_t*>(ks + Tile::kBytes + Tile::kCodeBytes) + gid;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 k = unpack2<__half>(km[8 * r]), v = unpack2<__half>(vm[8 * r]);
        const float sk = k.x * k_mul;
        x[i][2 * r] = fmaf(sk, x[i][2 * r], fmaf(k.y, qs0, -m0));
        x[i][2 * r + 1] = fmaf(sk, x[i][2 * r + 1], fmaf(k.y, qs1, -m1));
        sv[i][r] = v.x;
        mv[i][r] = v.y;
        if (MASK && 16 * i + 8 * r + gid >= valid) {
          x[i][2 * r] = x[i][2 * r + 1] = -INFINITY;
          sv[i][r] = mv[i][r] = 0.f;
        }
      }
      d0 = max3(d0, x[i][0], x[i][2]);
      d1 = max3(d1, x[i][1], x[i][3]);
      smax = max3(smax, fabsf(sv[i][0]), fabsf(sv[i][1]));
    }
    if (__any_sync(0xffffffffu, fmaxf(d0, d1) > limit || smax > cap))  // and before anything is summed: cap < 0
      move_reference<NB>(x, sv, smax);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      uint32_t p[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float e0 = exp2_approx(x[i][2 * r]), e1 = exp2_approx(x[i][2 * r + 1]);
        const float mid = fmaf(7.5f, sv[i][r], mv[i][r]);
        add2(l0, l1, e0, e1);
        fma2(b0, b1, e0, e1, mid, b0, b1);
        p[r] = pack2<__half>(e0 * sv[i][r], e1 * sv[i][r]);
      }
      p[0] = movmatrix_trans(p[0]);
      p[1] = movmatrix_trans(p[1]);
      mma_f16(ones, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, p[0], p[1]);
      pv(stage + (2 * i + 1) * Tile::kBytes, p[0], p[1], lane);
    }
    since_flush += NB;
    if (since_flush >= kFlushBlocks) flush();
  }

  // n (1..NB) consecutive blocks of a stage: whole stages as one step, a unit's
  // or share's last blocks one by one (masking a whole step instead, for the
  // sake of fewer steps, was no faster: 64 sequences 42.8 us against 41.8).
  template <int NB>
  __device__ __forceinline__ void blocks(const uint8_t* stage, int n, int valid, float scale_log2, int lane) {
    if (valid == 16 * NB) {
      step<NB, false>(stage, valid, scale_log2, lane);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; ++i) step<1, true>(stage + i * 2 * Tile::kBytes, valid - 16 * i, scale_log2, lane);
    }
  }

  __device__ __forceinline__ void finish_sums() {
    flush();
    l0 = sum_gid(l0);
    l1 = sum_gid(l1);
    b0 = sum_gid(b0);
    b1 = sum_gid(b1);
  }

  // Entries chunk_dim(lane, k) .. + 7 of head 2c + e, scaled by `mul`.
  __device__ __forceinline__ void chunk_values(int e, int k, float mul, float (&v)[8]) const {
    const float f = 16777216.f, h = 0.0625f * f, b = e ? b1 : b0;  // 2^24
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float(&even)[4] = acc[4 * k + 2 * w];
      const float(&odd)[4] = acc[4 * k + 2 * w + 1];
      v[4 * w] = fmaf(even[e], f, b) * mul;
      v[4 * w + 1] = fmaf(odd[e] - even[e], h, b) * mul;
      v[4 * w + 2] = fmaf(even[2 + e], f, b) * mul;
      v[4 * w + 3] = fmaf(odd[2 + e] - even[2 + e], h, b) * mul;
    }
  }
  __device__ __forceinline__ static int chunk_dim(int lane, int k) { return (D / 8) * (lane >> 2) + 8 * k; }
  static constexpr int kChunks = D / 64;
};

// ===================================================================== kernel

// A ring of kStages stages of up to kBlocksPerStage blocks per warp.  With the
// fused append, a unit's last stage holds a block less at most, and the
// appended token's K and V rows (fp16/bf16) take the last block's place.
template <int D>
struct Int4Shape {
  static constexpr int kWarps = 12;
  static constexpr int kBlocksPerStage = 4;
  static constexpr int kStages = 2;
  static constexpr int kBlockBytes = 2 * Int4Tile<D>::kBytes;  // K and V tile
  static constexpr int kStageBytes = kBlocksPerStage * kBlockBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
};

// Dynamic shared memory: [ring][prefix P[B+1]][context ctx[B]].
template <int D>
constexpr size_t int4_smem_bytes(int num_seqs) {
  return Int4Shape<D>::kRingBytes + (2 * static_cast<size_t>(num_seqs) + 1) * 4 + 128;
}
constexpr int kInt4MaxSeqs = 2048;
static_assert(int4_smem_bytes<128>(kInt4MaxSeqs) + 1536 <= 232448, "227 KB of shared memory, 1.5 KB kept for static");

// What a stage holds (written when it is issued, read when it is consumed).
struct StageInfo {
  static constexpr int kValidBits = 127;      // tokens of the context in it, 1..64
  static constexpr int kUnitStart = 1 << 7;   // its first block is the unit's first
  static constexpr int kUnitEnd = 1 << 8;     // its last block is the unit's last
  static constexpr int kShareStart = 1 << 9;  // the same for the share
  static constexpr int kShareEnd = 1 << 10;
  static constexpr int kCountShift = 11;      // blocks
};

// The fused append's patch of a unit's last stage: row r of the staged K and V
// tiles (at `tile`) and of the pool's (tile bytes at `off`) gets the new rows at
// `rows`, quantised.  D / 4 lanes take a row, four entries each (D = 64: both
// rows at once).
template <typename T, int D>
__device__ __forceinline__ void append_patch(uint8_t* tile, const uint8_t* rows, int r, uint8_t* k_pool,
                                             uint8_t* v_pool, int64_t off) {
  constexpr int W = D / 4;
  const int lane = threadIdx.x & 31, l = lane % W;
#pragma unroll
  for (int i = 0; i < W / 16; ++i) {
    const bool is_v = W == 32 ? i == 1 : lane >= 16;
    uint32_t pair;
    const uint32_t codes =
        int4_quantise4<T, W>(*reinterpret_cast<const uint2*>(rows + (is_v ? 2 * D : 0) + 8 * l), pair);
    int4_store4<D>(tile + (is_v ? Int4Tile<D>::kBytes : 0), is_v, r, l, codes, pair);
    if (off >= 0) int4_store4<D>((is_v ? v_pool : k_pool) + off, is_v, r, l, codes, pair);
  }
  fence_proxy_async_smem();  // the patch comes before the copies that refill the slot
  __syncwarp();
}

// Where the merge finds a unit's pieces.
struct UnitPieces {
  int32_t first;  // the share that it begins in, times two, + 1 if the piece is the share's second
  int32_t count;  // pieces, of that share and the next ones; 0: one share wrote it whole
};

// The shares: share w is blocks [w R, (w + 1) R) of the flattened space (cut off
// at `total`).  All of them are static: handing out their tails dynamically
// costs pieces to merge.  (64 x 16384 tokens 192.5 us with dynamic tails and
// 184.7 without, 256 x 4096 205.8 and 200.4; only from 2 GB a call on they are
// level, 512 x 4096 380.6 and 384.0, or better, 256 x 8192 370.7 and 383.)  A few
// blocks are a short step of work and pieces cost more than the warps they keep
// busy: a share is at least a 32nd of the average unit, up to kFew blocks, and
// never between half of kFew and kFew (1 x 8192 tokens 13.1 us, 14.5 with kFew 4
// and 15.7 with 16; 64 x 256 11.7, 13.4 and 13.4); and a unit has 256 pieces or
// so at most (one head of 131072 tokens 35.8 us, 55.3 without).
struct Int4Shares {
  static constexpr int kFew = 8;
  int total, R;
  __device__ __forceinline__ Int4Shares(int total_, int nwarps, int units) : total(total_), R(1) {
    if (total <= 0) return;
    const int average = total / units;
    R = max(max((total + nwarps - 1) / nwarps, min(kFew, average / 32)), average / 256);
    if (R > kFew / 2 && R < kFew) R = kFew;
  }
  __device__ __forceinline__ int start(int w) const { return min(total, w * R); }
};

// APPEND: the step, with k_new / v_new; else attention alone.  (One kernel for
// both cost attention 3.5 us of 39 at 8 x 16384 tokens.)
template <typename T, int D, bool APPEND>
__global__ void __maxnreg__(168) decode_int4_kernel(const DecodeArgs a) {
  using Tile = Int4Tile<D>;
  using Shape = Int4Shape<D>;
  using Attn = WarpAttnInt4<T, D>;
  constexpr int NW = Shape::kWarps, SW = Shape::kStages, NB = Shape::kBlocksPerStage;
  constexpr int kNewRowBytes = D * 2;  // one appended token's K (or V) row for one KV head (fp16/bf16)
  constexpr int kNewRows = (NB - 1) * Shape::kBlockBytes;  // where they lie in a unit's last stage
  static_assert(2 * kNewRowBytes <= Shape::kBlockBytes, "the appended rows fit one block");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[NW][SW];
  // (The share is the same for all of a warp's stages.  Read from here it costs no register: 16 x 2048 tokens 33.2 us,
  // and 33.9 with it kept, which spills.)
  __shared__ int4 s_desc[NW][SW];  // per stage: sequence, KV head, StageInfo, the warp's share
  __shared__ int s_prow[NW][SW];   // per stage: pool row of its last block (the fused append's target)
  __shared__ int s_warp_sum[NW];

  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  int* s_P = reinterpret_cast<int*>(ring + Shape::kRingBytes);
  int* s_ctx = s_P + a.num_seqs + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.num_seqs, Hkv = a.num_kv_heads, g = a.group;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int s = 0; s < SW; ++s) mbar_init(smem_u32(&full_bar[warp][s]), 1);
    fence_mbar_init();
  }
  // Lengths and tables read before the grid wait are a guess that is checked
  // after it, as in decode_persistent_kernel.
  context_prefix(a, a.pre_context_lens ? a.pre_context_lens : a.context_lens, s_P, s_ctx, s_warp_sum, NW * 32,
                 !a.recheck && blockIdx.x == 0);

  Int4Shares part(Hkv * s_P[B], gridDim.x * NW, B * Hkv);
  const int gw = blockIdx.x * NW + warp;

  // Sequence b, KV head kvh and block j of flattened block f: units are
  // ordered (b, kvh) and unit (b, kvh) holds blocks [Hkv*P[b] + kvh*nb, +nb).
  auto locate = [&](int f, int& b, int& kvh, int& j, int& nb) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (Hkv * s_P[mid] <= f) lo = mid; else hi = mid - 1;
    }
    b = lo;
    nb = (s_ctx[b] + kBlockSize - 1) / kBlockSize;
    const int rem = f - Hkv * s_P[b];
    kvh = rem / nb;
    j = rem - kvh * nb;
  };

  uint8_t* wring = ring + warp * SW * Shape::kStageBytes;
  const uint64_t policy = l2_evict_first_policy();

  const int32_t* tables = a.pre_block_tables ? a.pre_block_tables : a.block_tables;
  bool after_wait = !a.recheck;  // block ids are flagged only from values known to be final

  // ---- issue side: the share [share_s, share_e) and a 32-block window of it,
  // lane i describing block win_s + i.  The window is cut into stages at the
  // unit borders and every NB blocks (and before a unit's last block where the
  // appended rows would find no room): lane i's block belongs to stage
  // wstage, and the first lane of a stage holds its description.
  int share_s, share_e;
  int win_s, win_e;                  // window
  int stage_i = 0, stages = 0;       // next stage of the window to issue, and how many it has
  int wb = -1, wkvh = 0, wj = 0, wphys = -1, wrow = -kBlockSize, wstage = -1, wslot = 0, winfo = 0;
  bool bad_window = false;           // some block of the window is outside the pool
  auto fill_window = [&]() {
    win_s = win_e;
    win_e = min(share_e, win_s + 32);
    stage_i = 0;
    wb = -1; wkvh = 0; wj = 0; wphys = -1; wrow = -kBlockSize; wstage = -1; wslot = 0; winfo = 0;
    const int n = win_e - win_s;
    const bool in = lane < n;
    int nb = 0;
    if (in) {
      locate(win_s + lane, wb, wkvh, wj, nb);
      const int32_t* entry = tables + static_cast<int64_t>(wb) * a.max_blocks + wj;
      wphys = __ldcg(entry);
      if (wj == 0 || lane == 0)  // a unit starts here: bring its query rows into L2
        prefetch_l2_bulk(static_cast<const T*>(a.q) + (static_cast<int64_t>(wb) * Hkv + wkvh) * g * D,
                         static_cast<uint32_t>(g * D * sizeof(T)));
    }
    const unsigned upto = 0xffffffffu >> (31 - lane);
    const unsigned runs = __ballot_sync(0xffffffffu, in && (lane == 0 || wj == 0));
    const int pos = lane - (31 - __clz(runs & upto));  // lane 0 starts a run
    const unsigned firsts = __ballot_sync(
        0xffffffffu, in && (pos % NB == 0 || (APPEND && wj == nb - 1 && pos % NB == NB - 1)));
    stages = __popc(firsts);
    if (in) {
      wrow = tile_row(wphys, wkvh, a, after_wait);
      wstage = __popc(firsts & upto) - 1;
      wslot = lane - (31 - __clz(firsts & upto));
      const unsigned later = firsts & ~upto;
      const int count = (later ? __ffs(later) - 1 : n) - lane;  // blocks of the stage from this one on
      const int valid = min(count * kBlockSize, s_ctx[wb] - wj * kBlockSize);
      winfo = valid | (wj == 0 ? StageInfo::kUnitStart : 0) | (wj + count == nb ? StageInfo::kUnitEnd : 0) |
              (win_s + lane == share_s ? StageInfo::kShareStart : 0) |
              (win_s + lane + count == share_e ? StageInfo::kShareEnd : 0) | count << StageInfo::kCountShift;
    }
    bad_window = __any_sync(0xffffffffu, in && wrow < 0);
  };
  auto start_share = [&]() {
    share_s = part.start(gw);
    share_e = part.start(gw + 1);
    win_s = win_e = share_s;
    stage_i = stages = 0;
    if (win_e < share_e) fill_window();
  };

  int issued = 0, consumed = 0;
  int st_i = 0;            // stage slot the next issue fills
  int st_c = 0, ph_c = 0;  // stage slot the next consume reads, and its phase parity
  // Fill free stage slots; with may_advance false, up to the end of the window.
  auto issue_stages = [&](bool may_advance) {
    while (issued - consumed < SW) {
      if (stage_i == stages) {
        if (!may_advance || win_e >= share_e) break;
        fill_window();
      }
      const bool mine = wstage == stage_i;
      const uint32_t bar = smem_u32(&full_bar[warp][st_i]);
      uint8_t* stage = wring + st_i * Shape::kStageBytes;
      uint32_t bytes = (winfo >> StageInfo::kCountShift) * Shape::kBlockBytes;  // of the stage's first lane
      if (bad_window) {  // blocks outside the pool are not copied: they read as zeros
        const unsigned missing = __ballot_sync(0xffffffffu, mine && wrow < 0);
        bytes -= __popc(missing) * Shape::kBlockBytes;
        for (unsigned left = missing; left; left &= left - 1) {
          const int slot = __shfl_sync(0xffffffffu, wslot, __ffs(left) - 1);
          for (int o = lane * 16; o < Shape::kBlockBytes; o += 512)
            *reinterpret_cast<uint4*>(stage + slot * Shape::kBlockBytes + o) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // these writes come before the copies that refill the slot later
      }
      __syncwarp();  // every lane is done with this slot's last contents
      if (mine && wslot == 0) {
        s_desc[warp][st_i] = make_int4(wb, wkvh, winfo, gw);
        if (APPEND && (winfo & StageInfo::kUnitEnd)) {
          // A unit's last stage: the appended token's K and V rows too.
          const int64_t unit = static_cast<int64_t>(wb) * Hkv + wkvh;
          mbar_arrive_expect_tx(bar, bytes + 2 * kNewRowBytes);
          const uint32_t sd = smem_u32(stage + kNewRows);
          bulk_load(sd, static_cast<const T*>(a.k_new) + unit * D, kNewRowBytes, bar);
          bulk_load(sd + kNewRowBytes, static_cast<const T*>(a.v_new) + unit * D, kNewRowBytes, bar);
        } else {
          mbar_arrive_expect_tx(bar, bytes);
        }
      }
      if (APPEND && mine && winfo >> StageInfo::kCountShift == 1) s_prow[warp][st_i] = wrow;
      __syncwarp();  // the transaction count is set before the copies that complete it
      if (mine && wrow >= 0) {
        const uint32_t dst = smem_u32(stage) + wslot * Shape::kBlockBytes;
        const int64_t off = static_cast<int64_t>(wrow) * Tile::kRowBytes;
        bulk_load_hint(dst, static_cast<const uint8_t*>(a.k_cache_w) + off, Tile::kBytes, bar, policy);
        bulk_load_hint(dst + Tile::kBytes, static_cast<const uint8_t*>(a.v_cache_w) + off, Tile::kBytes, bar, policy);
      }
      ++issued;
      ++stage_i;
      st_i = st_i + 1 == SW ? 0 : st_i + 1;
    }
  };
  // Wait for the oldest stage in flight (bounded; false on a timeout).
  auto wait_oldest = [&]() -> bool { return mbar_wait(smem_u32(&full_bar[warp][st_c]), ph_c); };
  auto next_oldest = [&]() {
    ++consumed;
    if (++st_c == SW) {
      st_c = 0;
      ph_c ^= 1;
    }
  };

  // The share's first window (inputs only), its first stages' tiles prefetched
  // into L2, then the wait for the previous kernels in the stream.
  start_share();
  if (lane < SW * NB && win_s + lane < win_e && wrow >= 0) {
    const int64_t off = static_cast<int64_t>(wrow) * Tile::kRowBytes;
    prefetch_l2_bulk(static_cast<const uint8_t*>(a.k_cache_w) + off, Tile::kBytes);
    prefetch_l2_bulk(static_cast<const uint8_t*>(a.v_cache_w) + off, Tile::kBytes);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tables = a.block_tables;
  after_wait = true;

  // The first stages go out on the prologue's reading of the inputs; then the
  // lengths and this warp's first window of table entries are read again, and
  // if either changed the stages are dropped and everything is rebuilt from the
  // values read now.  With at most kWarpChecked sequences every warp compares
  // all the lengths itself once its first stage has landed; larger batches
  // compare at once with a CTA vote.  (decode_persistent_kernel has the reasons.)
  issue_stages(false);
  bool ok = true;
  if (a.recheck) {
    constexpr int kHeld = 4;
    constexpr int kWarpChecked = 32 * kHeld;
    const bool warp_check = B <= kWarpChecked;
    int held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      held[k] = warp_check && lane + 32 * k < B ? __ldcg(a.context_lens + lane + 32 * k) : 0;
    const bool in_window = win_s + lane < win_e;
    const int tv = in_window ? __ldcg(tables + static_cast<int64_t>(wb) * a.max_blocks + wj) : wphys;
    if (warp_check && issued > consumed) ok = wait_oldest();
    bool lens_changed;
    if (warp_check) {
      bool d = false;
      const bool flag = blockIdx.x == 0 && warp == 0;
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (lane + 32 * k < B) d |= clamp_context(held[k], a.max_blocks, flag) != s_ctx[lane + 32 * k];
      lens_changed = __any_sync(0xffffffffu, d);
    } else {
      lens_changed = context_changed(a, s_ctx, NW * 32, blockIdx.x == 0);
    }
    const bool table_changed = __any_sync(0xffffffffu, !lens_changed && in_window && tv != wphys);
    if (lens_changed || table_changed) {
      for (; ok && consumed < issued; next_oldest()) ok = wait_oldest();  // dropped, once they have landed
      if (lens_changed) {
        // CTA-uniform: every warp takes this branch.  The barrier keeps the
        // rebuild from changing s_ctx while another warp still compares.
        __syncthreads();
        context_prefix_again(a, s_P, s_ctx, s_warp_sum, NW * 32);
        part = Int4Shares(Hkv * s_P[B], gridDim.x * NW, B * Hkv);
      }
      start_share();
    } else if (in_window) {
      tile_row(wphys, wkvh, a, true);
    }
  }

  // What the merge will find of each unit, and zero rows for empty contexts.
  const int spread = warp * gridDim.x + blockIdx.x;  // a few warps of all CTAs
  for (int u = spread * 32 + lane; u < B * Hkv; u += gridDim.x * NW * 32) {
    const int b = u / Hkv, nb = (s_ctx[b] + kBlockSize - 1) / kBlockSize, U = Hkv * s_P[b] + (u - b * Hkv) * nb;
    const int w = U / part.R, n = nb > 0 ? (U + nb - 1) / part.R - w + 1 : 1;
    reinterpret_cast<UnitPieces*>(a.sched)[u] = {2 * w + (U > w * part.R ? 1 : 0), n > 1 ? n : 0};
  }
  for (int b = spread; b < B; b += gridDim.x * NW)
    if (s_ctx[b] == 0)
      for (int i = lane; i < a.num_q_heads * (D / 8); i += 32)
        reinterpret_cast<uint4*>(a.out)[static_cast<int64_t>(b) * a.num_q_heads * (D / 8) + i] = make_uint4(0, 0, 0, 0);

  // ---- consume side
  Attn at;
  bool from_start = false;   // the unit's blocks in this share begin with its first
  bool first_flush = true;   // of this share
  while (ok) {
    issue_stages(true);
    if (consumed == issued) break;
    __syncwarp();  // the descriptions written at issue are visible to the warp

    const int4 dsc = s_desc[warp][st_c];
    const int b = dsc.x, kvh = dsc.y, info = dsc.z, share = dsc.w;
    if (info & (StageInfo::kUnitStart | StageInfo::kShareStart)) {
      // While the tiles are under way: the query rows (L2), and a fresh state.
      from_start = info & StageInfo::kUnitStart;
      at.load_q(static_cast<const T*>(a.q) + (static_cast<int64_t>(b) * a.num_q_heads + kvh * g) * D, g, a.scale_log2,
                lane);
      at.reset();
    }
    if (!wait_oldest()) {  // timed out: flagged
      ok = false;
      break;
    }
    const int n = info >> StageInfo::kCountShift, valid = info & StageInfo::kValidBits;
    uint8_t* stage = wring + st_c * Shape::kStageBytes;
    if (APPEND && (info & StageInfo::kUnitEnd)) {
      // Append: the context's last token goes into its row of the stage's last
      // block, in the staged tiles (for this step's attention) and in the pool.
      const int prow = s_prow[warp][st_c];
      append_patch<T, D>(stage + (n - 1) * Shape::kBlockBytes, stage + kNewRows, (valid - 1) % kBlockSize,
                         static_cast<uint8_t*>(a.k_cache_w), static_cast<uint8_t*>(a.v_cache_w),
                         prow >= 0 ? static_cast<int64_t>(prow) * Tile::kRowBytes : -1);
    }
    at.template blocks<NB>(stage, n, valid, a.scale_log2, lane);
    next_oldest();

    if (info & (StageInfo::kUnitEnd | StageInfo::kShareEnd)) {
      // ---- the unit ends here or the share does: write it out, or leave a piece for the merge
      at.finish_sums();
      const int gid = lane >> 2, c = lane & 3;
      const bool complete = from_start && (info & StageInfo::kUnitEnd);
      const int64_t pbase = (static_cast<int64_t>(share) * 2 + (first_flush ? 0 : 1)) * kMaxGroup;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * c + e;
        if (h >= g) continue;
        const float l = e ? at.l1 : at.l0;
        if (complete) {
          T* orow = static_cast<T*>(a.out) + (static_cast<int64_t>(b) * a.num_q_heads + kvh * g + h) * D;
#pragma unroll
          for (int kk = 0; kk < Attn::kChunks; ++kk) {
            float v[8];
            at.chunk_values(e, kk, 1.f / l, v);
            *reinterpret_cast<uint4*>(orow + Attn::chunk_dim(lane, kk)) = pack8<T>(v);
          }
        } else {
          float* prow = a.part_o + (pbase + h) * D;
#pragma unroll
          for (int kk = 0; kk < Attn::kChunks; ++kk) {
            float v[8];
            at.chunk_values(e, kk, 1.f / l, v);
            float4* dst = reinterpret_cast<float4*>(prow + Attn::chunk_dim(lane, kk));
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
          if (gid == 0) a.part_lse[pbase + h] = (e ? at.m1 : at.m0) + log2f(l);
        }
      }
      first_flush = false;
    }
  }
  if (!ok && lane == 0) {
    // A wait gave up: let this warp's copies in flight land before the CTA exits.
    for (; consumed < issued; next_oldest()) wait_oldest();
  }
}

// ===================================================================== merge

// Merge of the units that shares cut.  S = 1: a warp per HN heads of a unit; S =
// kMergeWarps: a CTA per head, its warps every S-th piece.  A chain of two round
// trips to L2 after the decode grid's end (the description of the unit's pieces;
// the log-sum-exps together with the first pieces), where merge_persistent_kernel,
// which works the plan out from the lengths, takes four: no CTA of it fits beside
// a decode CTA (registers), so that nothing of it can be done before.
template <typename T, int D, int HN, int S>
__global__ void __launch_bounds__(kMergeWarps * 32, HN == 4 ? 4 : 8) merge_int4_kernel(const DecodeArgs a) {
  static_assert(S == 1 || (S == kMergeWarps && HN == 1), "several warps take one head");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kPer = D / 32, kFly = 8 / HN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = S == 1 ? 0 : warp;
  const int task = S == 1 ? blockIdx.x * kMergeWarps + warp : blockIdx.x;
  const int per = (a.group + HN - 1) / HN, unit = task / per, h0 = (task - unit * per) * HN;
  const int heads = HN == 1 ? 1 : min(HN, a.group - h0);
  const bool live = S > 1 || unit < a.num_seqs * a.num_kv_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 c = live ? __ldcg(reinterpret_cast<const int2*>(a.sched) + unit) : make_int2(0, 0);  // UnitPieces
  const int pieces = c.y;
  if (pieces == 0) return;
  const int n = (pieces - sub + S - 1) / S;  // this warp's
  auto row = [&](int i) {
    const int p = sub + S * i;
    return (p == 0 ? c.x : (c.x & ~1) + 2 * p) * kMaxGroup + h0;
  };
  float m[HN], L[HN], o[HN][kPer];
#pragma unroll
  for (int h = 0; h < HN; ++h) {
    m[h] = -INFINITY;
    L[h] = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[h][k] = 0.f;
  }
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int count = min(32, n - i0);
    float w[HN];
#pragma unroll
    for (int h = 0; h < HN; ++h)
      w[h] = lane < count && h < heads ? __ldcg(a.part_lse + row(i0 + lane) + h) : -INFINITY;
    for (int i = 0; i < count; i += kFly) {
      float v[kFly][HN][kPer];
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (i + u >= count) break;
        const float* src = a.part_o + static_cast<int64_t>(row(i0 + i + u)) * D + lane * kPer;
#pragma unroll
        for (int h = 0; h < HN; ++h) {  // (rows past the group's heads exist and are not used)
          if constexpr (kPer == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(src + h * D));
            v[u][h][0] = f.x, v[u][h][1] = f.y, v[u][h][2] = f.z, v[u][h][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(src + h * D));
            v[u][h][0] = f.x, v[u][h][1] = f.y;
          }
        }
      }
      if (i == 0) {  // the weights, with the first rows on their way
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          float mx = w[h];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          mx = fmaxf(mx, m[h]);
          const float sc = exp2f(m[h] - mx);
          m[h] = mx;
          w[h] = exp2f(w[h] - mx);
          float sum = w[h];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          L[h] = L[h] * sc + sum;
#pragma unroll
          for (int k = 0; k < kPer; ++k) o[h][k] *= sc;
        }
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (i + u >= count) break;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float wi = __shfl_sync(0xffffffffu, w[h], i + u);
#pragma unroll
          for (int k = 0; k < kPer; ++k) o[h][k] = fmaf(wi, v[u][h][k], o[h][k]);
        }
      }
    }
  }
  if constexpr (S > 1) {
    __shared__ float s_ml[S][2];
    __shared__ __align__(16) float s_o[S][D];
    if (lane == 0) {
      s_ml[sub][0] = m[0];
      s_ml[sub][1] = L[0];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) s_o[sub][lane * kPer + k] = o[0][k];
    __syncthreads();
    if (sub > 0) return;
    float mx = m[0];
#pragma unroll
    for (int s = 1; s < S; ++s) mx = fmaxf(mx, s_ml[s][0]);
    L[0] = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[0][k] = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const float sc = exp2f(s_ml[s][0] - mx);  // 0 for a warp without pieces
      L[0] = fmaf(s_ml[s][1], sc, L[0]);
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[0][k] = fmaf(s_o[s][lane * kPer + k], sc, o[0][k]);
    }
  }
  T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(unit) * a.group + h0) * D + lane * kPer;
#pragma unroll
  for (int h = 0; h < HN; ++h) {
    if (h < heads) {
      const float inv = 1.f / L[h];
#pragma unroll
      for (int k = 0; k < kPer; k += 2)
        *reinterpret_cast<uint32_t*>(out + h * D + k) = pack2<T>(o[h][k] * inv, o[h][k + 1] * inv);
    }
  }
}

}  // namespace pkv
