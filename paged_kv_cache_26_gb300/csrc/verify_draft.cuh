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
// memory; the warp whose piece holds the draw reads it again (from L2) to find
// the token.
#pragma once

#include "pkv_device.cuh"
#include "table_resize.cuh"

namespace pkv {

constexpr int kVerifyWarps = 16;
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

// A probability as a whole number of 2^-40; below 0 and NaN count as 0, above 1 as 1.
__device__ __forceinline__ unsigned long long prob_weight(float p) {
  return p > 0.f ? __float2ull_rn(fminf(p, 1.f) * 1099511627776.f) : 0ull;
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
  __shared__ int s_accepted, s_drafts;
  __shared__ unsigned long long s_warp[2][kVerifyWarps];  // [residual, p] sums of each warp's piece
  __shared__ unsigned long long s_total[2];               // of this CTA's, read by the cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster_size(), rank = cluster_rank();
  const int b = blockIdx.x / C, K = a.num_draft, V = a.vocab;
  const T* target = static_cast<const T*>(a.target) + b * a.target_seq;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.draft_seq : nullptr;

  const int ctx = a.context_lens ? a.context_lens[b] : 1;
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
    int n = a.draft_lens ? a.draft_lens[b] : K;
    bool bad = n < 0 || n > K;
    n = min(max(n, 0), K);
    bool ok = false;
    if (lane < n) {
      const int x = a.tokens[static_cast<int64_t>(b) * K + lane];
      if (x < 0 || x >= V) {
        bad = true;  // no such token: rejected
      } else {
        const double p = prob_value(target[lane * a.target_row + x]);
        const double q = draft ? prob_value(draft[lane * a.draft_row + x]) : 1.f;
        ok = static_cast<double>(a.accept_u[static_cast<int64_t>(b) * K + lane]) * q < p;
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
  auto weights = [&](int i, unsigned long long (&w)[4], unsigned long long (&wp)[4]) {
    float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
    load4<T>(prow, i, V, wide, p);
    if (qrow) load4<T>(qrow, i, V, wide, q);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      wp[k] = prob_weight(p[k]);
      const unsigned long long off = i + k == gone ? 1ull << kProbBits : prob_weight(q[k]);
      w[k] = wp[k] > off ? wp[k] - off : 0ull;
    }
  };
  unsigned long long sum = 0, sum_p = 0;
#pragma unroll 4
  for (int s = 0; s < steps; ++s) {
    const int i = first + s * 128 + lane * 4;
    if (i < V) {
      unsigned long long w[4], wp[4];
      weights(i, w, wp);
      sum += (w[0] + w[1]) + (w[2] + w[3]);
      sum_p += (wp[0] + wp[1]) + (wp[2] + wp[3]);
    }
  }
  sum = warp_sum(sum);
  sum_p = warp_sum(sum_p);
  if (lane == 0) s_warp[0][warp] = sum, s_warp[1][warp] = sum_p;
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
  const float uf = a.sample_u[b];
  const unsigned long long u = min(static_cast<unsigned long long>(uf > 0.f ? fminf(uf, 1.f) * 1073741824.f : 0.f),
                                   (1ull << kDrawBits) - 1);
  // floor(total u / 2^30): 62 + 30 bits
  const unsigned long long all = which ? total[1] : total[0];
  const unsigned long long goal = __umul64hi(all, u << (64 - kDrawBits));
  unsigned long long before = warp_sum(lane >= rank ? 0ull : which ? part[1] : part[0]);
  for (int w = 0; w < warp; ++w) before += s_warp[which][w];
  const unsigned long long mine = s_warp[which][warp];
  if (goal >= before && goal - before < mine) {  // one warp of the cluster (none if the total is 0)
    unsigned long long left = goal - before;
    for (int s = 0; s < steps; ++s) {
      const int i = first + s * 128 + lane * 4;
      unsigned long long w[4] = {0, 0, 0, 0}, wp[4] = {0, 0, 0, 0};
      if (i < V) weights(i, w, wp);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = which ? wp[k] : w[k];
      const unsigned long long own = (w[0] + w[1]) + (w[2] + w[3]);
      unsigned long long incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, left < incl);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          const unsigned long long r1 = incl - own + w[0], r2 = r1 + w[1], r3 = r2 + w[2];
          a.out_tokens[static_cast<int64_t>(b) * (K + 1) + acc] = i + (left >= r1) + (left >= r2) + (left >= r3);
        }
        break;
      }
      left -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (rank == 0) {
    if (tid <= K) {
      int32_t* out = a.out_tokens + static_cast<int64_t>(b) * (K + 1) + tid;
      if (tid < acc)
        *out = a.tokens[static_cast<int64_t>(b) * K + tid];
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
