// 4-bit KV cache (sm_103a): the format, its slot-mapped append and read-back.
// Decode attention over it is in decode_int4.cuh.
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

// Two float32 operations (each rounded to nearest even) in one instruction.
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {  // (x, y) += (a, b)
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 u, u, v;\n\t"
      "mov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// (x, y) = k (a, b) + (c, d)
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float k, float c, float d) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%5, %6};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 w, {%4, %4};\n\t"
      "fma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(k), "f"(c), "f"(d));
}

// The smaller / larger of two, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The stored pair of a row with these extremes (of values limited to the
// float16 range): m = f16(min), s = f16((max - m) / 15), all IEEE float32, so
// that the codes are the same wherever the formula is evaluated in float32.
// s rounds to 0 for a row of (nearly) equal values: its codes are then 0.
// A row with a NaN (both extremes are) has m = NaN, s = 0 and codes 0: it reads
// as NaN and attention that meets it gives NaN, as with a 16-bit pool.
struct Int4Row {
  float low, inv;
  uint32_t pair;  // scale in bits 0-15, minimum in bits 16-31
};
__device__ __forceinline__ Int4Row int4_row(float mn, float mx) {
  Int4Row r;
  const __half lo = __float2half_rn(mn);
  r.low = __half2float(lo);
  // The correctly rounded quotient by 15 from the product with the rounded 1/15
  // and one correction by the (exact) remainder (P. Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990); where a
  // step could underflow the quotient rounds to a float16 zero all the same.
  constexpr float kFifteenth = 1.f / 15.f;
  const float x = __fsub_rn(mx, r.low), y = __fmul_rn(x, kFifteenth);
  const __half sc = __float2half_rn(__fmaf_rn(__fmaf_rn(-15.f, y, x), kFifteenth, y));
  const float s = __half2float(sc);
  r.inv = s > 0.f ? __frcp_rn(s) : 0.f;
  if (mn != mn) {  // (x - low) * inv is then 0 or NaN for every x: code 0
    r.low = 0.f;
    r.inv = 0.f;
    r.pair = 0x7fffu << 16;
    return r;
  }
  r.pair = static_cast<uint32_t>(__half_as_ushort(sc)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
  return r;
}
__device__ __forceinline__ uint32_t int4_code(float x, const Int4Row& r) {
  const float v = rintf(__fmul_rn(__fsub_rn(x, r.low), r.inv));
  return static_cast<uint32_t>(fminf(fmaxf(v, 0.f), 15.f));  // a NaN gives 0
}
__device__ __forceinline__ float limit_f16(float x) { return min_nan(max_nan(x, -kF16Max), kF16Max); }

// One row of D values spread over W = D/4 neighbouring lanes, four consecutive
// values (packed in `raw`) each: the lane's four codes and the row's pair.
template <typename T, int W>
__device__ __forceinline__ uint32_t int4_quantise4(const uint2& raw, uint32_t& pair) {
  const float2 a = unpack2<T>(raw.x), b = unpack2<T>(raw.y);
  const float x0 = limit_f16(a.x), x1 = limit_f16(a.y), x2 = limit_f16(b.x), x3 = limit_f16(b.y);
  float mn = min_nan(min_nan(x0, x1), min_nan(x2, x3)), mx = max_nan(max_nan(x0, x1), max_nan(x2, x3));
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
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

// The larger / smaller of two packed pairs of T, half by half; NaN if either is.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (MmaKind<T>::kBf16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (MmaKind<T>::kBf16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 consecutive values of one row (packed), the row spread over L = D/16
// neighbouring lanes: their codes in order, eight to a word, and the row's pair.
// Extremes are found on the packed values (exact).  Codes need no limits, apart
// from rows told by `odd`: x - minimum is at least minus half a float16 step of
// the minimum, and the scale, if above 0, at least such a step, so the quotient
// is -0.5 or more and rounds to 0; the largest is checked once for the row.
// Rounding is by adding 1.5 * 2^23, which leaves the code in the low bits: a
// word is the sum of bits * 16^k, less what the upper bits add up to (mod 2^32).
template <typename T, int L>
__device__ __forceinline__ uint2 int4_quantise16(const uint4 (&raw)[2], uint32_t& pair) {
  uint32_t lo = word_of(raw[0], 0), hi = lo;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min2<T>(lo, word_of(raw[i >> 2], i & 3));
    hi = max2<T>(hi, word_of(raw[i >> 2], i & 3));
  }
  // One word holds (smallest, -largest): min2 reduces both at once.
  lo = min2<T>(lo, __byte_perm(lo, 0, 0x1032));
  hi = max2<T>(hi, __byte_perm(hi, 0, 0x1032)) ^ 0x80008000u;
  uint32_t ext = __byte_perm(lo, hi, 0x5410);
#pragma unroll
  for (int o = 1; o < L; o <<= 1) ext = min2<T>(ext, __shfl_xor_sync(0xffffffffu, ext, o));
  const float2 e = unpack2<T>(ext);
  const float mn = limit_f16(e.x), mx = limit_f16(-e.y);
  const Int4Row r = int4_row(mn, mx);
  pair = r.pair;
  constexpr float kMagic = 12582912.f;           // 1.5 * 2^23
  constexpr uint32_t kExcess = 0x4b400000u * 0x11111111u;  // its bits times 1 + 16 + .. + 16^7
  uint32_t out[2];
  // Values past the float16 range, a quotient that rounds above 15 (a scale in
  // float16's subnormal range), or a NaN (both extremes are): limited one by one.
  const bool odd = !(e.x >= -kF16Max && -e.y <= kF16Max && __fmul_rn(__fsub_rn(mx, r.low), r.inv) < 15.5f);
  if (odd) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      out[h] = 0;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const float2 x = unpack2<T>(word_of(raw[h], i));
        out[h] = out[h] << 8 | int4_code(limit_f16(x.y), r) << 4 | int4_code(limit_f16(x.x), r);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        float2 x = unpack2<T>(word_of(raw[h], i));
        add2(x.x, x.y, -r.low, -r.low);
        x.x = __fmul_rn(x.x, r.inv);  // (a packed product and sum would be fused to one rounding)
        x.y = __fmul_rn(x.y, r.inv);
        add2(x.x, x.y, kMagic, kMagic);
        w = w * 16 + __float_as_uint(x.y);
        w = w * 16 + __float_as_uint(x.x);
      }
      out[h] = w - kExcess;
    }
  }
  return make_uint2(out[0], out[1]);
}

constexpr int kAppendThreads = 256;
constexpr int kReadThreads = 256;

// Slot-mapped append into a 4-bit pool.  A CTA takes kAppendThreads / L
// neighbouring tokens of one KV head, L = D/16 lanes a row with 16 values each.
// V's codes of an even token and of the odd one after it share 32-bit words, so
// the lanes of an even token whose neighbour in the pool is the next token of
// the CTA (a prompt's tokens) take its codes through shared memory and store
// for both, whole words; other tokens store their 16-bit halves.
// Bound by the values read (2 bytes each) where tokens are many; 16 values a
// lane because the row's parameters (two divisions) and reductions are paid per
// lane.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
    append_int4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                       const int32_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int64_t num_slots,
                       uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int L = D / 16, kTokens = kAppendThreads / L;
  __shared__ int s_slot[kTokens + 1];
  __shared__ uint2 s_codes[kAppendThreads];
  const int tid = threadIdx.x, t = tid / L, l = tid % L;
  const int head = blockIdx.y;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + t;
  const bool in = token < num_tokens;
  int slot = in ? slots[token] : -1;
  uint4 kr[2] = {}, vr[2] = {};
  if (slot >= 0) {
    const int64_t at = ((token * num_kv_heads + head) * L + l) * 2;
    kr[0] = k_new[at], kr[1] = k_new[at + 1];
    vr[0] = v_new[at], vr[1] = v_new[at + 1];
  }
  if (slot >= num_slots) {
    if (l == 0) flag_error(kErrSlot);
    slot = -1;
  }
  uint32_t kp, vp;
  const uint2 kc = int4_quantise16<T, L>(kr, kp), vc = int4_quantise16<T, L>(vr, vp);
  if (l == 0) s_slot[t] = slot;
  if (tid == 0) s_slot[kTokens] = -1;
  s_codes[tid] = vc;
  __syncthreads();
  if (slot >= 0) {
    const int r = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * num_kv_heads + head) * Int4Tile<D>::kBytes;
    uint8_t* kt = k_cache + tile;
    uint8_t* vt = v_cache + tile;
    // K: quads in order, 8 bytes.
    *reinterpret_cast<uint2*>(kt + r * (D / 2) + 8 * l) = kc;
    if (l == 0) {
      *reinterpret_cast<uint32_t*>(kt + Int4Tile<D>::kCodeBytes + 4 * r) = kp;
      *reinterpret_cast<uint32_t*>(vt + Int4Tile<D>::kCodeBytes + 4 * r) = vp;
    }
    const bool leads = !(r & 1) && s_slot[t + 1] == slot + 1;
    const bool follows = (r & 1) && t > 0 && s_slot[t - 1] == slot - 1;
    if (leads) {
      const uint2 oc = s_codes[tid + L];
      const uint32_t w[4] = {__byte_perm(vc.x, oc.x, 0x5410), __byte_perm(vc.x, oc.x, 0x7632),
                             __byte_perm(vc.y, oc.y, 0x5410), __byte_perm(vc.y, oc.y, 0x7632)};
      if constexpr (D == 128) {
        *reinterpret_cast<uint4*>(vt + Int4Tile<D>::v_offset(r, 16 * l)) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<uint2*>(vt + Int4Tile<D>::v_offset(r, 16 * l)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(vt + Int4Tile<D>::v_offset(r, 16 * l + 8)) = make_uint2(w[2], w[3]);
      }
    } else if (!follows) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint16_t*>(vt + Int4Tile<D>::v_offset(r, 16 * l + 4 * i)) =
            static_cast<uint16_t>((i < 2 ? vc.x : vc.y) >> (16 * (i & 1)));
    }
  }
}

// Values of the rows at these slots, rounded to T: one thread reads dims 8c ..
// 8c + 7 of either half of a K row and of its V row (V's come with the
// neighbouring token's, in whole words).  A negative slot gives a zero row.
// Bound by the values written: so few lanes a row, as finding the tile and the
// pairs is paid per lane, and halves, as neighbouring lanes then store
// neighbouring 16 bytes.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads)
    read_int4_kernel(const int32_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int64_t num_slots,
                     const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                     uint4* __restrict__ k_out, uint4* __restrict__ v_out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int C = D / 16, kTokens = kReadThreads / C;
  const int c = threadIdx.x % C, head = blockIdx.y;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + threadIdx.x / C;
  if (token >= num_tokens) return;
  const int32_t slot = slots[token];
  uint4 kv[2][2] = {};
  if (slot >= num_slots) {
    if (c == 0) flag_error(kErrSlot);
  } else if (slot >= 0) {
    const int t = slot & 15;
    const int64_t tile = (static_cast<int64_t>(slot >> 4) * num_kv_heads + head) * Int4Tile<D>::kBytes;
    const uint8_t* kt = k_cache + tile;
    const uint8_t* vt = v_cache + tile;
    uint32_t kc[2];
    uint2 vw[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = 8 * c + j * (D / 2);
      kc[j] = *reinterpret_cast<const uint32_t*>(kt + t * (D / 2) + d / 2);
      vw[j] = *reinterpret_cast<const uint2*>(vt + Int4Tile<D>::v_offset(t & ~1, d));
    }
    const float2 ks = unpack2<__half>(*reinterpret_cast<const uint32_t*>(kt + Int4Tile<D>::kCodeBytes + 4 * t));
    const float2 vs = unpack2<__half>(*reinterpret_cast<const uint32_t*>(vt + Int4Tile<D>::kCodeBytes + 4 * t));
    const uint32_t pick = t & 1 ? 0x7632 : 0x5410;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t codes = v ? __byte_perm(vw[j].x, vw[j].y, pick) : kc[j];
        const float2 sm = v ? vs : ks;
        const uint32_t even = codes & 0x0f0f0f0fu, odd = codes >> 4 & 0x0f0f0f0fu;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // The code as the low byte of 2^23's bits; s * c is exact in float32
          // (11 + 4 bits): fused or not, one rounding.
          float x = __uint_as_float(__byte_perm(even, 0x4b000000u, 0x7650 + i));
          float y = __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7650 + i));
          add2(x, y, -8388608.f, -8388608.f);
          fma2(x, y, x, y, sm.x, sm.y, sm.y);
          w[i] = pack2<T>(x, y);
        }
        kv[v][j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  const int64_t at = (token * num_kv_heads + head) * (2 * C) + c;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    k_out[at + j * C] = kv[0][j];
    v_out[at + j * C] = kv[1][j];
  }
}

}  // namespace pkv
