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

}  // namespace pkv
