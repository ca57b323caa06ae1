// Verification of drafted tokens against the target's probabilities (sm_103a).
//
// Sequence b has n <= K drafted tokens x_0.., the target's distributions p_0 ..
// p_n and the draft's q_0 .. q_{n-1} (one-hot where it gives none).  Token i is
// accepted while u_i q_i(x_i) < p_i(x_i); the first one that is not is replaced
// by a draw from max(p_i - q_i, 0), and if all are accepted one more token is
// drawn from p_n.  The result is distributed as the target's own samples.
//
// A draw is the inverse CDF at a given u: the first token whose running sum
// exceeds u times the total.  Which token that is turns on the last bit of the
// sums, so the weights are whole numbers of 2^-40 (a float32 probability above
// 2^-17 is held exactly, a smaller one to within 2^-41), and the sums are exact
// in whatever order threads form them: the same token in every run, on every
// split of the row.  The acceptance compares the exact product, in float64.
//
// Bound by reading one row of p and, where a draft was rejected, one of q.  A
// cluster of CTAs shares a sequence's row, each warp a contiguous piece of it:
// 64-bit sums per warp, then per CTA, exchanged through distributed shared
// memory; the CTA that holds the draw reads the one piece it lies in again (from
// L2), all its warps together, to find the token.
#pragma once

#include "pkv_device.cuh"
#include "table_resize.cuh"

namespace pkv {

constexpr int kVerifyWarps = 8;
constexpr int kMaxVerifyCluster = 8;
constexpr int kMaxDrafts = 31;
constexpr int kProbBits = 40;    // weights are whole numbers of 2^-40
constexpr int kMaxVocab = 1 << 22;  // their sum stays below 2^62
constexpr int kDrawBits = 30;    // u as a whole number of 2^-30

struct VerifyArgs {
  const void* target;   // T[B][K + 1][V], strides below
  const void* draft;    // T[B][K][V] or null
  const int32_t* tokens;      // [B][K]
  const int32_t* draft_lens;  // [B] or null
  const float* accept_u;      // [B][K]
  const float* sample_u;      // [B]
  const int32_t* context_lens;  // [B] or null
  int32_t* num_accepted;      // [B]
  int32_t* out_tokens;        // [B][K + 1]
  int32_t* new_lens;          // [B] or null
  int64_t target_seq, target_row, draft_seq, draft_row;  // strides in elements
  int32_t num_draft, vocab;
};

__device__ __forceinline__ float prob_value(float v) { return v; }
__device__ __forceinline__ float prob_value(__half v) { return __half2float(v); }
__device__ __forceinline__ float prob_value(__nv_bfloat16 v) { return __bfloat162float(v); }

// A probability p in [0, 1] as a whole number w of 2^-40 (to nearest, half to
// even), in float32 operations and without a 64-bit conversion: adding 64
// rounds p to a multiple of 2^-17, h; p - h is exact, at most 2^-18, and its
// product with 2^40 is rounded by adding 1.5 * 2^23.  w = 2^23 (2^17 h) + low,
// the two whole numbers left in the sums' low bits, on top of constants.
constexpr uint32_t kHighBias = 0x42800000u;  // bits of 64
constexpr uint32_t kLowBias = 0x4b400000u;   // bits of 1.5 * 2^23
__device__ __forceinline__ void weight_parts(float p, uint32_t& high, uint32_t& low) {
  const float t = __fadd_rn(p, 64.f);
  const float r = __fsub_rn(p, __fsub_rn(t, 64.f));
  high = __float_as_uint(t);
  low = __float_as_uint(fmaf(r, 1099511627776.f, 12582912.f));
}
__device__ __forceinline__ unsigned long long prob_weight(float p) {
  uint32_t h, l;
  weight_parts(p, h, l);
  return (static_cast<unsigned long long>(h - kHighBias) << 23) + static_cast<long long>(static_cast<int32_t>(l - kLowBias));
}

// Four consecutive values from i on (those at or past V as 0).
template <typename T>
__device__ __forceinline__ void load4(const T* row, int i, int V, bool wide, float (&v)[4]) {
  if (wide && i + 3 < V) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row + i));
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(row + i));
      const float2 x = unpack2<T>(r.x), y = unpack2<T>(r.y);
      v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k < V ? prob_value(row[i + k]) : 0.f;
  }
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyWarps * 32) verify_draft_kernel(const VerifyArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int s_accepted, s_drafts;
  __shared__ unsigned long long s_warp[2][kVerifyWarps];  // [residual, p] sums of each warp's piece
  __shared__ unsigned long long s_total[2];               // of this CTA's, read by the cluster
  __shared__ unsigned long long s_scan[kVerifyWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster_size(), rank = cluster_rank();
  const int b = blockIdx.x / C, K = a.num_draft, V = a.vocab;
  const T* target = static_cast<const T*>(a.target) + b * a.target_seq;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.draft_seq : nullptr;

  // All that needs no other load first is asked for at once.
  const int ctx = a.context_lens ? a.context_lens[b] : 1;
  const float uf = a.sample_u[b];
  int n = K, x = -1;
  float accept = 0.f;
  if (warp == 0) {
    if (a.draft_lens) n = a.draft_lens[b];
    if (lane < K) {
      x = a.tokens[static_cast<int64_t>(b) * K + lane];
      accept = a.accept_u[static_cast<int64_t>(b) * K + lane];
    }
  }
  if (ctx <= 0) {  // an empty batch slot: nothing to verify (the same in every CTA of the cluster)
    if (rank == 0) {
      if (tid <= K) a.out_tokens[static_cast<int64_t>(b) * (K + 1) + tid] = -1;
      if (tid == 0) {
        a.num_accepted[b] = 0;
        if (a.new_lens) a.new_lens[b] = 0;
      }
    }
    return;
  }

  // ---- acceptance: lane i judges draft i
  if (warp == 0) {
    bool bad = n < 0 || n > K;
    n = min(max(n, 0), K);
    bool ok = false;
    if (lane < n) {
      if (x < 0 || x >= V) {
        bad = true;  // no such token: rejected
      } else {
        const double p = prob_value(target[lane * a.target_row + x]);
        const double q = draft ? prob_value(draft[lane * a.draft_row + x]) : 1.f;
        ok = static_cast<double>(accept) * q < p;
      }
    }
    const unsigned accepted = __ballot_sync(0xffffffffu, ok);
    if (bad && rank == 0) flag_error(kErrDraft);
    if (lane == 0) {
      s_accepted = __ffs(~accepted) - 1;  // at most K <= 31
      s_drafts = n;
    }
  }
  __syncthreads();
  const int acc = s_accepted;
  const bool rejected = acc < s_drafts;
  const T* prow = target + acc * a.target_row;
  const T* qrow = rejected && draft ? draft + acc * a.draft_row : nullptr;
  const int gone = rejected && !draft ? a.tokens[static_cast<int64_t>(b) * K + acc] : -1;  // q is one-hot there

  // ---- sums of this warp's piece of the row: steps of 128 entries
  const int pieces = C * kVerifyWarps, steps = (V + 128 * pieces - 1) / (128 * pieces);
  const int first = (rank * kVerifyWarps + warp) * steps * 128;
  constexpr uintptr_t kAlign = 4 * sizeof(T) - 1;
  const bool wide = ((reinterpret_cast<uintptr_t>(prow) | reinterpret_cast<uintptr_t>(qrow)) & kAlign) == 0;
  // Entries i..i+3 of p and of m = min(p, q), limited to [0, 1] (a NaN counts as
  // 0).  Weights are monotone, so max(w(p) - w(q), 0) = w(p) - w(m).
  const bool residual = rejected;
  auto load = [&](int i, float (&p)[4], float (&m)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = m[k] = 0.f;
    if (i < V) {
      load4<T>(prow, i, V, wide, p);
      if (qrow) load4<T>(qrow, i, V, wide, m);
    }
  };
  auto limit = [&](int i, float (&p)[4], float (&m)[4]) {  // (apart, so that loads can stay under way)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = __saturatef(p[k]);
      m[k] = fminf(p[k], i + k == gone ? 1.f : __saturatef(m[k]));
    }
  };
  long long sum_p = 0, sum_m = 0;
  // 8 entries a lane, and the next 8 on their way: within 64 registers, so that
  // four CTAs fit an SM (64 rows of 131072 entries 16.9 us; 16 entries without
  // the next on their way 19.6, with them, in 80 registers, 22.8).
  constexpr int kUnroll = 2;
  auto sum_up = [&](const float (&v)[kUnroll][4], long long& sum) {
    uint32_t high = 0, low = 0;  // the low parts' sum stays below 2^25
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h, l;
        weight_parts(v[u][k], h, l);
        high += h;
        low += l;
      }
    constexpr uint32_t n = 4 * kUnroll;
    sum += (static_cast<long long>(high - n * kHighBias) << 23) + static_cast<int32_t>(low - n * kLowBias);
  };
  auto at = [&](int s0, int u) { return s0 + u < steps ? first + (s0 + u) * 128 + lane * 4 : V; };
  auto fetch = [&](int s0, float (&p)[kUnroll][4], float (&m)[kUnroll][4]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(at(s0, u), p[u], m[u]);
  };
  auto add = [&](int s0, float (&p)[kUnroll][4], float (&m)[kUnroll][4]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) limit(at(s0, u), p[u], m[u]);
    sum_up(p, sum_p);
    if (residual) sum_up(m, sum_m);
  };
  float pa[kUnroll][4], ma[kUnroll][4], pb[kUnroll][4], mb[kUnroll][4];
  fetch(0, pa, ma);
  for (int s0 = 0; s0 < steps; s0 += 2 * kUnroll) {
    fetch(s0 + kUnroll, pb, mb);
    add(s0, pa, ma);
    fetch(s0 + 2 * kUnroll, pa, ma);
    add(s0 + kUnroll, pb, mb);
  }
  unsigned long long sum = sum_p - sum_m;
  sum = warp_sum(sum);
  const unsigned long long whole = warp_sum(sum_p);
  if (lane == 0) s_warp[0][warp] = sum, s_warp[1][warp] = whole;
  __syncthreads();
  if (tid < 2) {
    unsigned long long t = 0;
    for (int w = 0; w < kVerifyWarps; ++w) t += s_warp[tid][w];
    s_total[tid] = t;
  }
  cluster_sync();

  // ---- the draw: lane r holds CTA r's sums
  unsigned long long part[2] = {0, 0}, total[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (lane < C) {
      uint32_t remote;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(&s_total[k])), "r"(lane));
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(part[k]) : "r"(remote) : "memory");
    }
    total[k] = warp_sum(part[k]);
  }
  const int which = total[0] > 0 ? 0 : 1;  // nothing left of p - q (p <= q everywhere): from p itself
  const unsigned long long u = min(static_cast<unsigned long long>(uf > 0.f ? fminf(uf, 1.f) * 1073741824.f : 0.f),
                                   (1ull << kDrawBits) - 1);
  // floor(total u / 2^30): 62 + 30 bits
  const unsigned long long all = which ? total[1] : total[0];
  const unsigned long long goal = __umul64hi(all, u << (64 - kDrawBits));
  unsigned long long before = warp_sum(lane >= rank ? 0ull : which ? part[1] : part[0]);
  if (goal >= before && goal - before < s_total[which]) {  // one CTA of the cluster (none if the total is 0)
    int piece = 0;
    unsigned long long left = goal - before;
    for (; left >= s_warp[which][piece]; ++piece) left -= s_warp[which][piece];
    const int begin = (rank * kVerifyWarps + piece) * steps * 128;
    auto entry = [&](int i0) { return i0 + tid * 4 < steps * 128 ? begin + i0 + tid * 4 : V; };
    for (int i0 = 0; i0 < steps * 128; i0 += kVerifyWarps * 128) {
      const int i = entry(i0);
      float p[4], m[4];
      unsigned long long w[4];
      load(i, p, m);
      limit(i, p, m);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = prob_weight(p[k]) - (residual && !which ? prob_weight(m[k]) : 0ull);
      const unsigned long long own = (w[0] + w[1]) + (w[2] + w[3]);
      unsigned long long incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      __syncthreads();  // the previous pass's sums (and the first time s_warp's) have been read
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      unsigned long long run = incl - own, all_here = 0;
      for (int v = 0; v < kVerifyWarps; ++v) {
        const unsigned long long t = s_scan[v];
        if (v < warp) run += t;
        all_here += t;
      }
      if (left >= run && left - run < own) {
        const unsigned long long r1 = run + w[0], r2 = r1 + w[1], r3 = r2 + w[2];
        a.out_tokens[static_cast<int64_t>(b) * (K + 1) + acc] = i + (left >= r1) + (left >= r2) + (left >= r3);
      }
      if (left < all_here) break;  // the same in every thread
      left -= all_here;
    }
  }
  if (rank == 0) {
    if (tid <= K) {
      int32_t* out = a.out_tokens + static_cast<int64_t>(b) * (K + 1) + tid;
      if (tid < acc)
        *out = x;
      else if (tid > acc || all == 0)
        *out = -1;
    }
    if (tid == 0) {
      a.num_accepted[b] = acc;
      if (a.new_lens) a.new_lens[b] = max(ctx - (K - acc), 0);
    }
  }
  cluster_sync();  // the sums stay readable until every CTA has read them
}

}  // namespace pkv
