// 4-bit KV cache (sm_103a): the format, its slot-mapped append, the read-back,
// and one warp's attention over 4-bit tiles (run by decode_persistent_kernel).
//
// A row (one token of one KV head, D values) is held as codes c in 0..15 and a
// float16 pair (scale s, minimum m): value = s * c + m.  The 16 rows of a
// (block, KV head) form one contiguous tile of 16 * (D/2 + 4) bytes: the
// codes, then the 16 pairs.  One untiled bulk copy brings a tile in whole, so
// the byte order inside it is free and is the one the mma fragments want,
// without a swizzle and without bank conflicts:
//   K codes: row-major, dims d and d + 1 in byte d/2 (low four bits first).
//     Lane (gid = lane/4, c = lane%4) reads the c-th quarter of rows gid and
//     gid + 8: 32 lanes x 16 bytes in a row.
//   V codes: the four codes (16 bits) of dims 4i..4i+3 of an even token and of
//     the odd token after it lie side by side in one 32-bit word, so masking a
//     word gives the two tokens of one dim that an mma A register holds.  With
//     G = D/8 dims per gid: byte (t/8) 4D + (d/G) 4G + (t/2 % 4) G +
//     (d%G)/4 * 4 + (t%2) 2 + (d%4)/2; lane (gid, c) reads G consecutive bytes
//     of either half, again 32 lanes in a row.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

template <int D>
struct Int4Tile {
  static constexpr int kCodeBytes = 8 * D;        // 16 rows of D/2 bytes
  static constexpr int kBytes = kCodeBytes + 64;  // + 16 (scale, minimum) pairs
  static constexpr int kRowBytes = D / 2 + 4;     // kBytes / 16
  static constexpr int kDimsPerGid = D / 8;
  // Byte of V's codes of dims d..d+3 (d a multiple of 4) of token t: 2 bytes.
  __device__ __forceinline__ static int v_offset(int t, int d) {
    constexpr int G = kDimsPerGid;
    return (t >> 3) * (4 * D) + (d / G) * (4 * G) + ((t >> 1) & 3) * G + (d % G) + (t & 1) * 2;
  }
};

constexpr float kF16Max = 65504.f;

// The stored pair of a row with these extremes (of values limited to the
// float16 range): m = f16(min), s = f16((max - m) / 15), all IEEE float32, so
// that the codes are the same wherever the formula is evaluated in float32.
// s rounds to 0 for a row of (nearly) equal values: its codes are then 0.
struct Int4Row {
  float low, inv;
  uint32_t pair;  // scale in bits 0-15, minimum in bits 16-31
};
__device__ __forceinline__ Int4Row int4_row(float mn, float mx) {
  Int4Row r;
  const __half lo = __float2half_rn(mn);
  r.low = __half2float(lo);
  const __half sc = __float2half_rn(__fdiv_rn(__fsub_rn(mx, r.low), 15.f));
  const float s = __half2float(sc);
  r.inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  r.pair = static_cast<uint32_t>(__half_as_ushort(sc)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
  return r;
}
__device__ __forceinline__ uint32_t int4_code(float x, const Int4Row& r) {
  const float v = rintf(__fmul_rn(__fsub_rn(x, r.low), r.inv));
  return static_cast<uint32_t>(fminf(fmaxf(v, 0.f), 15.f));  // a NaN gives 0
}
__device__ __forceinline__ float limit_f16(float x) { return fminf(fmaxf(x, -kF16Max), kF16Max); }

// One row of D values spread over W = D/4 neighbouring lanes, four consecutive
// values (packed in `raw`) each: the lane's four codes and the row's pair.
template <typename T, int W>
__device__ __forceinline__ uint32_t int4_quantise4(const uint2& raw, uint32_t& pair) {
  const float2 a = unpack2<T>(raw.x), b = unpack2<T>(raw.y);
  const float x0 = limit_f16(a.x), x1 = limit_f16(a.y), x2 = limit_f16(b.x), x3 = limit_f16(b.y);
  float mn = fminf(fminf(x0, x1), fminf(x2, x3)), mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const Int4Row r = int4_row(mn, mx);
  pair = r.pair;
  return int4_code(x0, r) | int4_code(x1, r) << 4 | int4_code(x2, r) << 8 | int4_code(x3, r) << 12;
}

// Store the four codes of lane l (of W) and, from l == 0, the pair of token t
// of a K (is_v false) or V tile.
template <int D>
__device__ __forceinline__ void int4_store4(uint8_t* tile, bool is_v, int t, int l, uint32_t codes, uint32_t pair) {
  const int off = is_v ? Int4Tile<D>::v_offset(t, 4 * l) : t * (D / 2) + 2 * l;
  *reinterpret_cast<uint16_t*>(tile + off) = static_cast<uint16_t>(codes);
  if (l == 0) *reinterpret_cast<uint32_t*>(tile + Int4Tile<D>::kCodeBytes + 4 * t) = pair;
}

// ===================================================================== append

// Slot-mapped append into a 4-bit pool: a warp quantises one token's K and V
// rows of one KV head (D = 64: one half-warp each).
template <typename T, int D>
__global__ void append_int4_kernel(const uint2* __restrict__ k_new, const uint2* __restrict__ v_new,
                                   const int32_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads,
                                   int64_t num_slots, uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int W = D / 4;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t row = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5); row < rows;
       row += warps) {
    const int64_t token = row / num_kv_heads;
    const int head = static_cast<int>(row - token * num_kv_heads);
    const int32_t slot = slots[token];
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (lane == 0) flag_error(kErrSlot);
      continue;
    }
    const int t = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * num_kv_heads + head) * Int4Tile<D>::kBytes;
    const int l = lane % W;
#pragma unroll
    for (int h = 0; h < W / 16; ++h) {
      const bool is_v = W == 32 ? h == 1 : lane >= 16;
      const uint2 raw = (is_v ? v_new : k_new)[row * W + l];
      uint32_t pair;
      const uint32_t codes = int4_quantise4<T, W>(raw, pair);
      int4_store4<D>((is_v ? v_cache : k_cache) + tile, is_v, t, l, codes, pair);
    }
  }
}

// Values of the rows at these slots, rounded to T: one thread reads eight dims
// of a K row and of its V row.  A negative slot gives a zero row.
template <typename T, int D>
__global__ void read_int4_kernel(const int32_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads,
                                 int64_t num_slots, const uint8_t* __restrict__ k_cache,
                                 const uint8_t* __restrict__ v_cache, uint4* __restrict__ k_out,
                                 uint4* __restrict__ v_out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int C = D / 8;
  const int64_t total = static_cast<int64_t>(num_tokens) * num_kv_heads * C;
  for (int64_t idx = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = idx / C;
    const int d = static_cast<int>(idx - row * C) * 8;
    const int64_t token = row / num_kv_heads;
    const int head = static_cast<int>(row - token * num_kv_heads);
    const int32_t slot = slots[token];
    if (slot < 0 || slot >= num_slots) {
      if (slot >= num_slots) flag_error(kErrSlot);
      k_out[idx] = v_out[idx] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const int t = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * num_kv_heads + head) * Int4Tile<D>::kBytes;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      const uint8_t* p = (is_v ? v_cache : k_cache) + tile;
      uint32_t codes;
      if (is_v) {
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(p + Int4Tile<D>::v_offset(t, d));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(p + Int4Tile<D>::v_offset(t, d + 4));
        codes = lo | hi << 16;
      } else {
        codes = *reinterpret_cast<const uint32_t*>(p + t * (D / 2) + d / 2);
      }
      const float2 sm = unpack2<__half>(*reinterpret_cast<const uint32_t*>(p + Int4Tile<D>::kCodeBytes + 4 * t));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // s * c is exact in float32 (11 + 4 bits): fused or not, one rounding
        w[i] = pack2<T>(fmaf(static_cast<float>(codes >> (8 * i) & 15u), sm.x, sm.y),
                        fmaf(static_cast<float>(codes >> (8 * i + 4) & 15u), sm.x, sm.y));
      (is_v ? v_out : k_out)[idx] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ===================================================================== warp math

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One warp's attention state for one (sequence, KV head) unit over 4-bit tiles.
//
// Codes go to the tensor cores without a conversion: a code masked out of its
// word in place, c or 16 c in the low bits of a 16-bit half, is the float16
// subnormal c * 2^-24 or c * 2^-20, which mma.sync multiplies exactly.  Eight
// codes cost one shift and four ANDs.
//   scores:  q . K_t = s_t (q . c_t) + m_t sum(q)            (float32, per token)
//   output:  sum_t p_t V_t = sum_t P_t c_t + sum_t p_t m_t,  P_t = p_t s_t
// P is rounded to float16 relative to R, the power of two at or below the
// largest scale met so far, so that small scales keep their bits.  The
// rounding must act on c - 7.5 and not on c, whose common part is several
// times the value: with a = sum of the rounded P,
//   sum_t P_t c_t + sum_t p_t m_t = [sum P_t c_t - 7.5 a] + sum_t p_t (m_t + 7.5 s_t).
// The bracket is formed every kFlushBlocks blocks (flush), which also keeps
// the accumulators at the output's size: an accumulator that carried 7.5 a
// over a long context would lose the output's low bits to it.
//
// Lane (gid = lane/4, c = lane%4): scores of tokens gid, gid + 8 and heads 2c,
// 2c + 1 as in WarpAttn; O^T entries of dims [G gid, G gid + G), G = D/8.
template <typename T, int D>
struct WarpAttnInt4 {
  using Tile = Int4Tile<D>;
  static constexpr int kWords = D / 32;  // 32-bit words of codes per lane and row
  static constexpr int kFlushBlocks = 64;
  uint32_t qf[4 * kWords];
  float acc[D / 16][4];
  float m0, m1, l0, l1;  // running max (log2 units) and sum of p
  float a0, a1, b0, b1;  // sums of rounded P since the last flush, and of p (m + 7.5 s)
  float qs0, qs1;        // scale_log2 * sum(q)
  float ref;             // R
  int since_flush;

  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = a0 = a1 = b0 = b1 = 0.f;
    ref = 5.9604644775390625e-8f;  // 2^-24, the smallest float16 scale
    since_flush = 0;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }

  // Entries [(D/4) c, (D/4) (c + 1)) of query row gid as float16 in the order
  // the masked K words pair them; a bf16 query beyond the float16 range is
  // flagged (kErrQuery).  Word w holds dims d0..d7: registers (d0,d4), (d2,d6)
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

  static constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

  // 2^-24 (q . c) of tokens gid (x[0..1]) and gid + 8 (x[2..3]), heads 2c, 2c + 1.
  __device__ __forceinline__ void dots(const uint8_t* ks, int lane, float (&x)[4]) const {
    uint32_t wa[kWords], wb[kWords];
    load_words(ks + lane * (D / 8), wa);               // row gid, quarter c: (4 gid + c) D/8
    load_words(ks + Tile::kCodeBytes / 2 + lane * (D / 8), wb);  // row gid + 8
    float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t ya = wa[w] >> 8, yb = wb[w] >> 8;
      mma16816<__half>(s, wa[w] & kLow, wb[w] & kLow, ya & kLow, yb & kLow, qf[4 * w], qf[4 * w + 1]);
      mma16816<__half>(t, wa[w] & kHigh, wb[w] & kHigh, ya & kHigh, yb & kHigh, qf[4 * w + 2], qf[4 * w + 3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaf(t[i], 0.0625f, s[i]);
  }

  // acc += V^T P^T for one tile: m-tile 2w + h holds dims 4w + h (rows gid) and
  // 4w + h + 2 (rows gid + 8) of the lane's G, times 2^-24 (h = 0) or 2^-20.
  __device__ __forceinline__ void pv(const uint8_t* vs, uint32_t p0, uint32_t p1, int lane) {
    uint32_t x[kWords], y[kWords];
    load_words(vs + lane * (D / 8), x);                          // tokens 2c, 2c + 1
    load_words(vs + Tile::kCodeBytes / 2 + lane * (D / 8), y);   // tokens 2c + 8, 2c + 9
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t x8 = x[w] >> 8, y8 = y[w] >> 8;
      mma16816<__half>(acc[2 * w], x[w] & kLow, x8 & kLow, y[w] & kLow, y8 & kLow, p0, p1);
      mma16816<__half>(acc[2 * w + 1], x[w] & kHigh, x8 & kHigh, y[w] & kHigh, y8 & kHigh, p0, p1);
    }
  }

  // Sum over the lanes that share c.
  __device__ __forceinline__ static float sum_gid(float v) {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  __device__ __forceinline__ void flush() {
    const float f0 = sum_gid(a0) * (7.5f * 5.9604644775390625e-8f), f1 = sum_gid(a1) * (7.5f * 5.9604644775390625e-8f);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float u = i & 1 ? 16.f : 1.f;
      acc[i][0] -= u * f0;
      acc[i][1] -= u * f1;
      acc[i][2] -= u * f0;
      acc[i][3] -= u * f1;
    }
    a0 = a1 = 0.f;
    since_flush = 0;
  }

  // Accumulate n (1..NB) consecutive blocks of one unit as one softmax step;
  // their (K tile, V tile) pairs lie back to back at `stage`, and the first
  // `valid` (1..16 n) tokens belong to the context.  Pairs and codes of slots
  // past `valid` may hold anything: their scores and scales are replaced.
  template <int NB>
  __device__ __forceinline__ void blocks(const uint8_t* stage, int n, int valid, float scale_log2, int lane) {
    const int gid = lane >> 2;
    const float k_mul = scale_log2 * 16777216.f;  // 2^24
    float x[NB][4], sv[NB][2], mv[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      x[i][0] = x[i][1] = x[i][2] = x[i][3] = -INFINITY;
      sv[i][0] = sv[i][1] = mv[i][0] = mv[i][1] = 0.f;
      if (i < n) {
        const uint8_t* ks = stage + i * 2 * Tile::kBytes;
        float d[4];
        dots(ks, lane, d);
        const uint32_t* km = reinterpret_cast<const uint32_t*>(ks + Tile::kCodeBytes);
        const uint32_t* vm = reinterpret_cast<const uint32_t*>(ks + Tile::kBytes + Tile::kCodeBytes);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (16 * i + 8 * r + gid < valid) {
            const float2 k = unpack2<__half>(km[gid + 8 * r]), v = unpack2<__half>(vm[gid + 8 * r]);
            const float sk = k.x * k_mul;
            x[i][2 * r] = fmaf(sk, d[2 * r], k.y * qs0);
            x[i][2 * r + 1] = fmaf(sk, d[2 * r + 1], k.y * qs1);
            sv[i][r] = v.x;
            mv[i][r] = v.y;
          }
        }
      }
    }
    float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]), smax = fmaxf(fabsf(sv[0][0]), fabsf(sv[0][1]));
#pragma unroll
    for (int i = 1; i < NB; ++i) {
      mx0 = fmaxf(mx0, fmaxf(x[i][0], x[i][2]));
      mx1 = fmaxf(mx1, fmaxf(x[i][1], x[i][3]));
      smax = fmaxf(smax, fmaxf(fabsf(sv[i][0]), fabsf(sv[i][1])));
    }
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
    }
    // The largest scale's exponent (the bits of a float >= 0 order as it does).
    const float r_new = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(smax)) & 0x7f800000u);
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);  // finite: token 0 is valid
    // The rescale is skipped while neither a maximum nor the reference moves.
    if (__any_sync(0xffffffffu, mn0 > m0 || mn1 > m1 || r_new > ref)) {
      const float al0 = exp2_approx(m0 - mn0), al1 = exp2_approx(m1 - mn1);
      const float f = r_new > ref ? ref / r_new : 1.f;
      const float g0 = al0 * f, g1 = al1 * f;
      ref = fmaxf(ref, r_new);
      m0 = mn0;
      m1 = mn1;
      l0 *= al0;
      l1 *= al1;
      b0 *= al0;
      b1 *= al1;
      a0 *= g0;
      a1 *= g1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        acc[i][0] *= g0;
        acc[i][1] *= g1;
        acc[i][2] *= g0;
        acc[i][3] *= g1;
      }
    }
    const float inv_ref = 1.f / ref;  // exact: a power of two
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (i < n) {
        uint32_t p[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float e0 = exp2_approx(x[i][2 * r] - m0), e1 = exp2_approx(x[i][2 * r + 1] - m1);
          const float s = sv[i][r] * inv_ref, mid = fmaf(7.5f, sv[i][r], mv[i][r]);
          l0 += e0;
          l1 += e1;
          b0 = fmaf(e0, mid, b0);
          b1 = fmaf(e1, mid, b1);
          p[r] = pack2<__half>(e0 * s, e1 * s);
          const float2 pr = unpack2<__half>(p[r]);
          a0 += pr.x;
          a1 += pr.y;
        }
        pv(stage + (2 * i + 1) * Tile::kBytes, movmatrix_trans(p[0]), movmatrix_trans(p[1]), lane);
      }
    }
    since_flush += n;
    if (since_flush >= kFlushBlocks) flush();
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
    const float f = ref * 16777216.f, b = e ? b1 : b0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float(&even)[4] = acc[4 * k + 2 * w];
      const float(&odd)[4] = acc[4 * k + 2 * w + 1];
      v[4 * w] = fmaf(even[e], f, b) * mul;
      v[4 * w + 1] = fmaf(odd[e], 0.0625f * f, b) * mul;
      v[4 * w + 2] = fmaf(even[2 + e], f, b) * mul;
      v[4 * w + 3] = fmaf(odd[2 + e], 0.0625f * f, b) * mul;
    }
  }
  __device__ __forceinline__ static int chunk_dim(int lane, int k) { return (D / 8) * (lane >> 2) + 8 * k; }
  static constexpr int kChunks = D / 64;
};

}  // namespace pkv
