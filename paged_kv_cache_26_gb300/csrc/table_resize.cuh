// Block tables and slot maps from the sequences' lengths, on the GPU (sm_103a).
//
// Every sequence goes from context_lens[b] to new_lens[b] tokens.  With n(L) =
// ceil(L / 16) blocks, sequence b takes n(new) - n(old) blocks or gives back
// n(old) - n(new).  All positions follow from three prefix sums over the
// sequences (tokens gained, blocks taken, blocks given), so no thread waits
// for another's result:
//   * the free list is a stack of `count` ids.  Given blocks go on first, the
//     r-th (in order of sequence and block) at count + R - 1 - r, R their
//     number; then the i-th taken comes off at count + R - 1 - i.  Growing and
//     shrinking back therefore leaves the list as it was.  A position at or
//     past count is read from the giver's table row, which nobody writes;
//   * slot s of the map belongs to the sequence whose gained tokens straddle s
//     (binary search), and its block is either in the table already or the
//     taken block of known rank.
// The work is latency: a few kilobytes for a decode step, 4 bytes per gained
// token for prompts.  One cluster of CTAs does it in one launch: each CTA forms
// the prefix sums by itself (cheaper than handing them round), they share the
// output, and the lengths and the count are overwritten in place only after
// the cluster's barrier, when every CTA has read them.
#pragma once

#include <climits>

#include "paged_kv_kernels.cuh"
#include "pkv_device.cuh"

namespace pkv {

constexpr int kResizeThreads = 1024;  // at most
constexpr int kResizeCluster = 16;    // CTAs for prompts
constexpr int kSlotRun = 16;          // slots a thread writes at a time, at most
constexpr int kMaxResizeSeqs = 8192;  // four int32 arrays in shared memory

struct ResizeArgs {
  int32_t* context_lens;
  const int32_t* new_lens;
  int32_t* block_tables;
  int32_t* free_blocks;
  int32_t* num_free;
  int32_t* slot_mapping;   // may be null
  int32_t* token_offsets;  // may be null
  int32_t num_seqs, max_blocks, num_blocks, num_slots;
};

inline size_t resize_smem_bytes(int num_seqs) { return (4 * static_cast<size_t>(num_seqs) + 3) * sizeof(int32_t); }

// Largest b in [0, n) with pre[b] <= x, for pre ascending from 0 and x < pre[n]:
// the sequence that holds element x (sequences with nothing are passed over).
__device__ __forceinline__ int holder(const int* pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the barrier wants whole warps
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__global__ void __launch_bounds__(kResizeThreads, 1) resize_tables_kernel(const ResizeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ int resize_smem[];
  __shared__ long long s_wtok[32];
  __shared__ int s_wtake[32], s_wgive[32];
  const int B = a.num_seqs, MB = a.max_blocks;
  int* s_old = resize_smem;      // [B]
  int* s_tok = s_old + B;        // [B + 1] tokens gained before sequence b
  int* s_take = s_tok + B + 1;   // [B + 1] blocks taken
  int* s_give = s_take + B + 1;  // [B + 1] blocks given
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank();
  const int cta = blockDim.x, warps = cta / 32;
  const int nthreads = cluster_size() * cta, gtid = rank * cta + tid;

  // ---- prefix sums: each thread takes `per` consecutive sequences
  const int per = (B + cta - 1) / cta;
  const int lo = min(B, tid * per), hi = min(B, lo + per);
  const int count = *a.num_free;
  long long tok = 0;
  int take = 0, give = 0, bad = 0;
  for (int b = lo; b < hi; ++b) {
    const int old = a.context_lens[b], now = a.new_lens[b];
    bad |= old < 0 || old > MB * kBlockSize || now < 0 || now > MB * kBlockSize;
    const int d = (now + kBlockSize - 1) / kBlockSize - (old + kBlockSize - 1) / kBlockSize;
    s_old[b] = old;
    s_tok[b] = max(now - old, 0);
    s_take[b] = max(d, 0);
    s_give[b] = max(-d, 0);
    tok += s_tok[b];
    take += s_take[b];
    give += s_give[b];
  }
  long long itok = tok;
  int itake = take, igive = give;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, itok, o);
    const int u = __shfl_up_sync(0xffffffffu, itake, o), v = __shfl_up_sync(0xffffffffu, igive, o);
    if (lane >= o) itok += t, itake += u, igive += v;
  }
  if (lane == 31) s_wtok[warp] = itok, s_wtake[warp] = itake, s_wgive[warp] = igive;
  bad = __syncthreads_or(bad);
  long long btok = itok - tok, total_tok = 0;
  int btake = itake - take, bgive = igive - give, T = 0, R = 0;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    if (w < warp) btok += s_wtok[w], btake += s_wtake[w], bgive += s_wgive[w];
    total_tok += s_wtok[w], T += s_wtake[w], R += s_wgive[w];
  }
  for (int b = lo; b < hi; ++b) {
    const int t = s_tok[b], u = s_take[b], v = s_give[b];
    s_tok[b] = static_cast<int>(btok), s_take[b] = btake, s_give[b] = bgive;
    btok += t, btake += u, bgive += v;
  }
  if (tid == 0) s_tok[B] = static_cast<int>(total_tok), s_take[B] = T, s_give[B] = R;
  __syncthreads();

  // ---- all or nothing: every CTA reaches the same verdict
  unsigned err = bad ? kErrContext : 0;
  if (!bad) {
    if (count < 0 || count > a.num_blocks || static_cast<long long>(count) + R - T > a.num_blocks)
      err = kErrFreeList;
    else if (static_cast<long long>(count) + R < T)
      err = kErrNoBlocks;
    else if (total_tok > (a.slot_mapping ? a.num_slots : INT_MAX))
      err = kErrSlot;
  }
  if (err) {
    if (gtid == 0) flag_error(err);
    if (a.slot_mapping)
      for (int i = gtid; i < a.num_slots; i += nthreads) a.slot_mapping[i] = -1;
    if (a.token_offsets)
      for (int i = gtid; i <= B; i += nthreads) a.token_offsets[i] = 0;
    return;  // the same in every CTA of the cluster
  }
  const int top = count + R;  // the stack's height once the given blocks are on it
  auto table = [&](int b, int j) -> int32_t* { return a.block_tables + static_cast<int64_t>(b) * MB + j; };
  // Block at this position of the stack.
  auto at_position = [&](int pos) -> int {
    int id;
    if (pos < count) {
      id = a.free_blocks[pos];
    } else {
      const int r = top - 1 - pos, b = holder(s_give, B, r);
      const int nb_old = (s_old[b] + kBlockSize - 1) / kBlockSize;
      id = *table(b, nb_old - (s_give[b + 1] - r));
    }
    return id;
  };

  // ---- the slots of the gained tokens: each thread a run of them, for which one
  // search, and mostly one or two blocks, will do; single slots while they are
  // few, since then the time is one thread's chain of loads
  if (a.slot_mapping) {
    const int total = static_cast<int>(total_tok);
    const bool wide = (reinterpret_cast<uintptr_t>(a.slot_mapping) & 15) == 0;
    const int run = a.num_slots <= nthreads ? 1 : a.num_slots <= 4 * nthreads ? 4 : kSlotRun;
    for (int64_t i0 = static_cast<int64_t>(gtid) * run; i0 < a.num_slots; i0 += static_cast<int64_t>(nthreads) * run) {
      const int begin = static_cast<int>(i0), end = static_cast<int>(min(i0 + run, static_cast<int64_t>(a.num_slots)));
      int b = begin < total ? holder(s_tok, B, begin) : 0, held = -1, base = -1;
      // First slot of block j of sequence b, or -1.
      auto find = [&](int j) {
        if (j == held) return;
        const int nb_old = (s_old[b] + kBlockSize - 1) / kBlockSize;
        const int id = j < nb_old ? *table(b, j) : at_position(top - 1 - (s_take[b] + j - nb_old));
        if (id < 0 || id >= a.num_blocks) flag_error(kErrBlockId);
        base = id < 0 || id >= a.num_blocks ? -1 : id * kBlockSize;
        held = j;
      };
      for (int i = begin; i < end; i += 4) {
        int v[4] = {-1, -1, -1, -1};
        const int pos = s_old[b] + (i - s_tok[b]);
        if (i + 4 <= min(end, s_tok[b + 1]) && pos % kBlockSize <= kBlockSize - 4) {  // four of one block
          find(pos / kBlockSize);
          if (base >= 0)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = base + pos % kBlockSize + k;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (i + k >= min(end, total)) break;
            if (i + k >= s_tok[b + 1]) {
              do ++b;
              while (i + k >= s_tok[b + 1]);
              held = -1;
            }
            const int at = s_old[b] + (i + k - s_tok[b]);
            find(at / kBlockSize);
            v[k] = base < 0 ? -1 : base + at % kBlockSize;
          }
        }
        if (wide && i + 4 <= end && run > 1) {
          *reinterpret_cast<int4*>(a.slot_mapping + i) = make_int4(v[0], v[1], v[2], v[3]);
        } else {
          for (int k = 0; k < 4 && i + k < end; ++k) a.slot_mapping[i + k] = v[k];
        }
      }
    }
  }

  // ---- table entries of the taken blocks, and the given blocks that stay on the list
  // (four at a time: their searches and loads overlap)
  constexpr int kIlp = 4;
  for (int i0 = gtid; i0 < T; i0 += kIlp * nthreads) {
    int id[kIlp], b[kIlp];
#pragma unroll
    for (int k = 0; k < kIlp; ++k) {
      const int i = i0 + k * nthreads;
      b[k] = i < T ? holder(s_take, B, i) : 0;
      id[k] = i < T ? at_position(top - 1 - i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kIlp; ++k) {
      const int i = i0 + k * nthreads;
      if (id[k] < 0 || id[k] >= a.num_blocks) flag_error(kErrBlockId);
      if (i < T) *table(b[k], (s_old[b[k]] + kBlockSize - 1) / kBlockSize + i - s_take[b[k]]) = id[k];
    }
  }
  for (int r0 = T + gtid; r0 < R; r0 += kIlp * nthreads) {
    int id[kIlp];
#pragma unroll
    for (int k = 0; k < kIlp; ++k) {
      const int r = r0 + k * nthreads;
      id[k] = r < R ? at_position(top - 1 - r) : 0;
    }
#pragma unroll
    for (int k = 0; k < kIlp; ++k) {
      const int r = r0 + k * nthreads;
      if (id[k] < 0 || id[k] >= a.num_blocks) flag_error(kErrBlockId);
      if (r < R) a.free_blocks[top - 1 - r] = id[k];
    }
  }
  if (a.token_offsets)
    for (int i = gtid; i <= B; i += nthreads) a.token_offsets[i] = s_tok[i];

  cluster_sync();  // every CTA has read the lengths and the count
  for (int b = gtid; b < B; b += nthreads) a.context_lens[b] = a.new_lens[b];
  if (gtid == 0) *a.num_free = top - T;
}

}  // namespace pkv
