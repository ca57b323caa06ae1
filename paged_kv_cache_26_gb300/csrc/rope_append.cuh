// Rotary positions (sm_103a): rows of queries and keys turned to their tokens'
// positions, the keys and values stored at their slots of a paged cache on the
// way (or the keys written out as rows).
//
// Frequency f turns its pair of dims (i, j) by the angle a = position * w_f:
//   x'_i = x_i cos a - x_j sin a,   x'_j = x_j cos a + x_i sin a,
// with (i, j) = (f, f + rot/2), or (2f, 2f + 1) when interleaved; dims past rot
// stay.  A token has up to four positions (time, height, width, ...), of which
// every frequency takes one.
//
// Angles.  Only the fraction of a turn matters, and float32 loses it at far
// positions (position 10^6 at w = 1: a float32 product is good to 0.06 rad).  So a
// frequency is held as turns per position in units of 2^-64, a 64-bit integer made by
// a float64 product (off by 2^-52 of itself and the 2^-64 cut off): position * turns
// modulo 2^64 is the fraction, off by that times the position and by nothing else.
// Its upper 32 bits, signed, are half turns in [-1, 1), and as a float32 for sincospif
// right to 2^-26 of a turn.  Three integer multiplications instead of float64
// arithmetic.
//
// Bound by the bytes of the rows: 16,384 tokens of 32 + 8 + 8 heads, D = 128, bf16 (403
// MB in and out) take 68 us, 5.9 TB/s.  A CTA takes up to four tokens, makes their sines
// and cosines once in shared memory (every head shares them), its first rows already
// on their way, and then treats all rows alike, two 16-byte vectors a thread and step:
// the eight pairs of eight neighbouring frequencies.  (Eight tokens a CTA 70 us, sixteen
// 75, the next step's loads ahead of this one's stores 75: fewer threads fit.)  The same
// tokens into E4M3 pools (369 MB) 70 us, 5.3 TB/s; rows to rows (336 MB) 59 us, 5.7 TB/s.
#pragma once

#include "paged_kv_kernels.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // tokens of a CTA, at most
constexpr int kMaxFreqs = 64;

struct RopeArgs {
  const void* q;  // T[tokens][Hq][D] with strides, or null (no query rows)
  const void* k;
  const void* v;  // null: no value rows
  void* q_out;
  void* k_out;              // rows, or the K pool
  void* v_out;              // the V pool
  const int32_t* positions; // [axes][tokens]
  const int32_t* slots;     // pools only
  const float* k_scale;     // E4M3 pools only
  const float* v_scale;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // strides in 16-byte units
  int64_t qo_token, qo_head, ko_token, ko_head;
  int64_t num_slots;
  int32_t num_tokens, num_q_heads, num_kv_heads;
  int32_t head_vecs;        // 16-byte vectors of a row: D / 8
  int32_t freqs;            // rot / 2, a multiple of 8
  int32_t interleaved;
  int32_t tokens_per_cta;
  uint32_t row_magic;       // ceil(2^32 / rows of a token): exact quotients of numbers below 2^16
  float factor;             // multiplies sine and cosine
  uint64_t axis_bits[2];    // two bits a frequency: its position axis
  uint64_t turns[kMaxFreqs];
};

enum RopeDst : int { kRopeRows, kRopePool16, kRopePoolE4M3 };

template <typename T>
__device__ __forceinline__ void rotate8(uint4& x, uint4& y, const float2* cs, bool interleaved) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<T>(word_of(x, i)), w = unpack2<T>(word_of(y, i));
    if (interleaved) {  // x: pairs 0..3, y: pairs 4..7
      a[i] = u.x;
      b[i] = u.y;
      a[4 + i] = w.x;
      b[4 + i] = w.y;
    } else {
      a[2 * i] = u.x;
      a[2 * i + 1] = u.y;
      b[2 * i] = w.x;
      b[2 * i + 1] = w.y;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 t = cs[i];  // (cos, sin)
    const float ra = fmaf(a[i], t.x, -(b[i] * t.y)), rb = fmaf(b[i], t.x, a[i] * t.y);
    a[i] = ra;
    b[i] = rb;
  }
  if (interleaved) {
    x = make_uint4(pack2<T>(a[0], b[0]), pack2<T>(a[1], b[1]), pack2<T>(a[2], b[2]), pack2<T>(a[3], b[3]));
    y = make_uint4(pack2<T>(a[4], b[4]), pack2<T>(a[5], b[5]), pack2<T>(a[6], b[6]), pack2<T>(a[7], b[7]));
  } else {
    x = make_uint4(pack2<T>(a[0], a[1]), pack2<T>(a[2], a[3]), pack2<T>(a[4], a[5]), pack2<T>(a[6], a[7]));
    y = make_uint4(pack2<T>(b[0], b[1]), pack2<T>(b[2], b[3]), pack2<T>(b[4], b[5]), pack2<T>(b[6], b[7]));
  }
}

template <typename T, int DST>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 s_cs[kRopeTokens * kMaxFreqs];
  __shared__ int64_t s_slot[kRopeTokens];
  const int t0 = blockIdx.x * a.tokens_per_cta;
  const int nt = min(a.tokens_per_cta, a.num_tokens - t0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int pairs = a.head_vecs >> 1;                 // steps of two vectors in a row: 4 or 8
  const int shift = pairs == 8 ? 3 : 2;
  const int rows = a.num_q_heads + (a.v ? 2 : 1) * a.num_kv_heads;
  const int rot = a.freqs >> 3;                       // steps that turn; the others copy
  const int total = nt * rows << shift;

  struct Step {
    int t, h, kind, j;  // kind 0: query, 1: key, 2: value
    int64_t lo, hi;     // the two vectors, from the row's start
  };
  auto locate = [&](int i) {
    Step s;
    s.j = i & (pairs - 1);
    const uint32_t r = static_cast<uint32_t>(i) >> shift;
    s.t = static_cast<int>(__umulhi(r, a.row_magic));
    if (rows == 1) s.t = static_cast<int>(r);         // (the magic of 1 is 2^32)
    s.h = static_cast<int>(r) - s.t * rows;
    s.kind = 0;
    if (s.h >= a.num_q_heads) {
      s.h -= a.num_q_heads;
      s.kind = 1;
      if (s.h >= a.num_kv_heads) {
        s.h -= a.num_kv_heads;
        s.kind = 2;
      }
    }
    if (s.kind != 2 && s.j < rot && !a.interleaved) {
      s.lo = s.j;
      s.hi = s.j + rot;
    } else {  // neighbours: interleaved pairs, dims past rot, values
      s.lo = 2 * s.j;
      s.hi = 2 * s.j + 1;
    }
    return s;
  };
  auto load = [&](const Step& s, uint4& x, uint4& y) {
    const uint4* p = s.kind == 0   ? static_cast<const uint4*>(a.q) + (t0 + s.t) * a.q_token + s.h * a.q_head
                     : s.kind == 1 ? static_cast<const uint4*>(a.k) + (t0 + s.t) * a.k_token + s.h * a.k_head
                                   : static_cast<const uint4*>(a.v) + (t0 + s.t) * a.v_token + s.h * a.v_head;
    x = p[s.lo];
    y = p[s.hi];
  };
  Step s0 = locate(min(static_cast<int>(threadIdx.x), total - 1)), s1 = locate(min(static_cast<int>(threadIdx.x) + kRopeThreads, total - 1));
  uint4 x0, y0, x1, y1;
  load(s0, x0, y0);
  load(s1, x1, y1);
  for (int i = threadIdx.x; i < nt * a.freqs; i += kRopeThreads) {
    const int t = i / a.freqs, f = i - t * a.freqs;
    const int axis = static_cast<int>(a.axis_bits[f >> 5] >> (2 * (f & 31))) & 3;
    const int64_t pos = a.positions[static_cast<int64_t>(axis) * a.num_tokens + t0 + t];
    const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[f];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    s_cs[t * a.freqs + f] = make_float2(c * a.factor, s * a.factor);
  }
  if (DST != kRopeRows && threadIdx.x < static_cast<unsigned>(nt)) {
    int64_t slot = a.slots[t0 + threadIdx.x];
    if (slot >= a.num_slots) {
      flag_error(kErrSlot);
      slot = -1;
    }
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();

  auto store = [&](const Step& s, uint4 x, uint4 y) {
    if (s.kind != 2 && s.j < rot) rotate8<T>(x, y, s_cs + s.t * a.freqs + 8 * s.j, a.interleaved);
    if (s.kind == 0 || DST == kRopeRows) {
      uint4* p = s.kind == 0 ? static_cast<uint4*>(a.q_out) + (t0 + s.t) * a.qo_token + s.h * a.qo_head
                             : static_cast<uint4*>(a.k_out) + (t0 + s.t) * a.ko_token + s.h * a.ko_head;
      p[s.lo] = x;
      p[s.hi] = y;
      return;
    }
    const int64_t slot = s_slot[s.t];
    if (slot < 0) return;
    const int64_t row = ((slot >> 4) * a.num_kv_heads + s.h) * kBlockSize + (slot & 15);
    void* pool = s.kind == 1 ? a.k_out : a.v_out;
    if constexpr (DST == kRopePool16) {
      uint4* p = static_cast<uint4*>(pool) + row * a.head_vecs;
      p[s.lo] = x;
      p[s.hi] = y;
    } else {
      const float scale = __ldg((s.kind == 1 ? a.k_scale : a.v_scale) + s.h);
      uint2* p = static_cast<uint2*>(pool) + row * a.head_vecs;
      p[s.lo] = quantize8<T>(x, scale);  // of the row as T holds it: the codes of an append of turned rows
      p[s.hi] = quantize8<T>(y, scale);
    }
  };
  for (int i = threadIdx.x; i < total;) {
    store(s0, x0, y0);
    if (i + kRopeThreads < total) store(s1, x1, y1);
    i += 2 * kRopeThreads;
    if (i >= total) break;
    s0 = locate(i);
    s1 = locate(min(i + kRopeThreads, total - 1));
    load(s0, x0, y0);
    load(s1, x1, y1);
  }
}

}  // namespace pkv
