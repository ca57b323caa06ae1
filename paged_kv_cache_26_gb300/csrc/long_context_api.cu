// C ABI of the operators around prompts and long contexts: rotary positions and
// the append that turns its keys, attention of chunks of new tokens, and decode
// over the blocks that the bounds of their keys select.  The declarations and
// their contracts are in include/paged_kv.h.
#include "pkv_host.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <limits>

#include "block_select.cuh"
#include "chunk_attention.cuh"
#include "pkv_internal.h"
#include "rope_append.cuh"

namespace {

// Devices on which this unit has launched a kernel: elsewhere its error word is 0 and
// paged_kv_check_status need not read it (a copy of its own, 23 us with both against 14).
// A captured launch counts from its capture on.
std::atomic<bool> g_launched[kMaxDevices];

template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), dim3 grid, unsigned cluster, unsigned threads, size_t smem,
                   cudaStream_t stream, Args... args) {
  g_launched[current_device()].store(true, std::memory_order_relaxed);
  return launch_dependent(kern, grid, cluster, threads, smem, stream, args...);
}

// f(T) for the value type of d.
template <typename F>
void with_type(const pkv_dims* d, F&& f) {
  d->dtype == PKV_DTYPE_BF16 ? f(__nv_bfloat16{}) : f(__half{});
}

// ------------------------------------------------------------------ rotary positions

int rope_impl(const void* q, const void* k, const void* v, const int32_t* positions, const int32_t* slots,
              int32_t num_tokens, const pkv_rope* rope, void* q_out, void* k_out, void* v_out, const float* k_scale,
              const float* v_scale, const pkv_rope_strides* strides, const pkv_dims* d, int dst, const char* name,
              cudaStream_t stream) {
  const std::string what = name;
  int rc = check_dims(d, false);
  if (rc != PKV_OK) return rc;
  if (!rope) return pkv_fail(PKV_ERR_INVALID_ARG, what + ": rope is NULL");
  if (num_tokens < 0 || d->num_q_heads < 0) return pkv_fail(PKV_ERR_INVALID_ARG, what + ": negative size");
  if (rope->rot_dim < 16 || rope->rot_dim > d->head_dim || rope->rot_dim % 16 != 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": rot_dim must be a multiple of 16, at most head_dim");
  if (rope->num_axes < 1 || rope->num_axes > 4)
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": 1 to 4 position axes");
  for (int f = 0; f < rope->rot_dim / 2; ++f)
    if (static_cast<int>(rope->axis_bits[f >> 5] >> (2 * (f & 31)) & 3) >= rope->num_axes)
      return pkv_fail(PKV_ERR_INVALID_ARG, what + ": a frequency's axis is not among num_axes");
  const int64_t rows = static_cast<int64_t>(d->num_q_heads) + (dst == pkv::kRopeRows ? 1 : 2) * static_cast<int64_t>(d->num_kv_heads);
  if (rows > 8192) return pkv_fail(PKV_ERR_UNSUPPORTED, what + ": more than 8192 rows a token");
  if (num_tokens == 0) return PKV_OK;
  const bool queries = d->num_q_heads > 0;
  if (!k || !positions || !k_out || (queries && (!q || !q_out)))
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": NULL pointer");
  if (dst != pkv::kRopeRows && (!v || !v_out || !slots || (dst == pkv::kRopePoolE4M3 && (!k_scale || !v_scale))))
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": NULL pointer");
  const uintptr_t pool = dst == pkv::kRopePoolE4M3 ? 8 : 16;
  if (!aligned(k, 16) || !aligned(k_out, dst == pkv::kRopeRows ? 16 : pool) || !aligned(v_out, pool) ||
      !aligned(v, 16) || (queries && (!aligned(q, 16) || !aligned(q_out, 16))) || !aligned(positions, 4) ||
      !aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": misaligned pointer (rows and 16-bit pools need 16 bytes)");
  pkv_rope_strides s = {};
  if (strides) {
    s = *strides;
    for (const int64_t x : {s.q_token, s.q_head, s.k_token, s.k_head, s.v_token, s.v_head, s.q_out_token, s.q_out_head,
                            s.k_out_token, s.k_out_head})
      if (x < 0 || x % 8 != 0)
        return pkv_fail(PKV_ERR_INVALID_ARG, what + ": strides must be multiples of 8 elements and not negative");
  } else {
    const int64_t D = d->head_dim;
    s.q_head = s.k_head = s.v_head = s.q_out_head = s.k_out_head = D;
    s.q_token = s.q_out_token = d->num_q_heads * D;
    s.k_token = s.v_token = s.k_out_token = d->num_kv_heads * D;
  }
  pkv::RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = dst == pkv::kRopeRows ? nullptr : v;
  a.q_out = q_out;
  a.k_out = k_out;
  a.v_out = v_out;
  a.positions = positions;
  a.slots = slots;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.q_token = s.q_token / 8;
  a.q_head = s.q_head / 8;
  a.k_token = s.k_token / 8;
  a.k_head = s.k_head / 8;
  a.v_token = s.v_token / 8;
  a.v_head = s.v_head / 8;
  a.qo_token = s.q_out_token / 8;
  a.qo_head = s.q_out_head / 8;
  a.ko_token = s.k_out_token / 8;
  a.ko_head = s.k_out_head / 8;
  a.num_slots = static_cast<int64_t>(d->num_blocks) * pkv::kBlockSize;
  a.num_tokens = num_tokens;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.head_vecs = d->head_dim / 8;
  a.freqs = rope->rot_dim / 2;
  a.interleaved = rope->interleaved != 0;
  // Tokens share the latency of their sines: as few a CTA as make one round of CTAs, four
  // on an SM, and four where there are more rounds (1,500 tokens, 32 + 8 + 8 heads: three
  // 9.4 us, two 10.4; 2,000: four 11.4, two 12.7).
  a.tokens_per_cta = 1;
  while (a.tokens_per_cta < pkv::kRopeTokens && num_tokens > static_cast<int64_t>(a.tokens_per_cta) * 4 * device_sms())
    ++a.tokens_per_cta;
  a.row_magic = static_cast<uint32_t>(((int64_t(1) << 32) + rows - 1) / rows);
  a.factor = rope->factor;
  a.axis_bits[0] = rope->axis_bits[0];
  a.axis_bits[1] = rope->axis_bits[1];
  std::copy(rope->turns, rope->turns + a.freqs, a.turns);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(num_tokens) + a.tokens_per_cta - 1) / a.tokens_per_cta);
  cudaError_t e = cudaSuccess;
  with_type(d, [&](auto t) {
    using T = decltype(t);
    auto kern = dst == pkv::kRopeRows     ? pkv::rope_kernel<T, pkv::kRopeRows>
                : dst == pkv::kRopePool16 ? pkv::rope_kernel<T, pkv::kRopePool16>
                                          : pkv::rope_kernel<T, pkv::kRopePoolE4M3>;
    e = launch(kern, dim3(grid), 1, pkv::kRopeThreads, 0, stream, a);
  });
  if (e != cudaSuccess) return cuda_fail(e, "rope_kernel launch");
  return PKV_OK;
}

// ------------------------------------------------------------------ shared checks

int check_tables(const pkv_dims* d, const void* block_tables, const void* context_lens, const std::string& what) {
  if (!context_lens || (!block_tables && d->max_blocks_per_seq > 0))
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": NULL pointer");
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, what + ": misaligned pointer");
  if (static_cast<int64_t>(d->max_blocks_per_seq) * pkv::kBlockSize >= (int64_t(1) << 31))
    return pkv_fail(PKV_ERR_UNSUPPORTED, what + ": max_blocks_per_seq * 16 must be < 2^31");
  return PKV_OK;
}

// ------------------------------------------------------------------ chunks of new tokens

// Two partial results for each CTA of the grid, then how each CTA's part begins.
size_t chunk_partials(const pkv_dims* d) {
  return align256(static_cast<size_t>(2) * device_sms() * pkv::kChunkRows * (d->head_dim + 2) * sizeof(float));
}
size_t chunk_workspace(const pkv_dims* d) {
  return chunk_partials(d) + align256(device_sms() * sizeof(pkv::ChunkCut));
}

// Queries as (dims, heads, tokens): a box is 64 dims of the group's heads of a
// tile's tokens, which lie in shared memory as rows of 128 bytes, a token's heads
// side by side.
int make_query_map(CUtensorMap* map, const void* q, int32_t num_tokens, const pkv_dims* d, int group) {
  auto fn = encode_fn();
  if (!fn) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d->head_dim), static_cast<cuuint64_t>(d->num_q_heads),
                              static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d->head_dim) * 2,
                                 static_cast<cuuint64_t>(d->num_q_heads) * d->head_dim * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, d->dtype == PKV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        3, const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(r) + ")");
  return PKV_OK;
}

// A pool as (64 dims, 8 tokens, D / 64, groups of 8 tokens): the box of a block puts
// the atoms of its two groups one after the other (beside ChunkShape).
int make_block_map(CUtensorMap* map, const void* cache, const pkv_dims* d) {
  auto fn = encode_fn();
  if (!fn) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t row = static_cast<cuuint64_t>(d->head_dim) * 2;
  const cuuint32_t parts = static_cast<cuuint32_t>(d->head_dim / 64);
  const cuuint64_t dims[4] = {64, 8, parts, static_cast<cuuint64_t>(d->num_blocks) * d->num_kv_heads * 2};
  const cuuint64_t strides[3] = {row, 128, 8 * row};
  const cuuint32_t box[4] = {64, 8, parts, 2};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, d->dtype == PKV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(r) + ")");
  return PKV_OK;
}

int chunk_attention_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                         const int32_t* context_lens, const int32_t* q_offsets, int32_t num_tokens, float scale,
                         void* out, void* workspace, size_t workspace_bytes, const pkv_dims* d, cudaStream_t stream) {
  int rc = check_dims(d, true);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return pkv_fail(PKV_ERR_INVALID_ARG, "chunk_attention: num_tokens < 0");
  if (!std::isfinite(scale)) return pkv_fail(PKV_ERR_INVALID_ARG, "chunk_attention: scale is not finite");
  if (d->num_seqs > pkv::kMaxChunkSeqs)
    return pkv_fail(PKV_ERR_UNSUPPORTED,
                    "chunk_attention: at most " + std::to_string(pkv::kMaxChunkSeqs) + " sequences per call");
  if (d->num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if ((rc = check_tables(d, block_tables, context_lens, "chunk_attention")) != PKV_OK) return rc;
  if (!q || !k_cache || !v_cache || !q_offsets || !out) return pkv_fail(PKV_ERR_INVALID_ARG, "chunk_attention: NULL pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(q_offsets, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, "chunk_attention: misaligned pointer (q/out/caches need 16 bytes)");
  const size_t need = chunk_workspace(d);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
    return pkv_fail(PKV_ERR_INVALID_ARG, "chunk_attention: workspace missing, too small (" + std::to_string(need) +
                                             " bytes needed) or not 256-byte aligned");
  if (d->max_blocks_per_seq > (1 << 26))
    return pkv_fail(PKV_ERR_UNSUPPORTED, "chunk_attention: at most 2^26 blocks a table");
  // The line of work is counted in 64 bits.  (Offsets that fall may give many sequences
  // all of the rows.)
  const double keys = d->num_seqs * (num_tokens / 32.0 + 1) * (16.0 * d->max_blocks_per_seq + num_tokens + 256.0) * d->num_kv_heads;
  if (keys > 4e18) return pkv_fail(PKV_ERR_UNSUPPORTED, "chunk_attention: too many tokens, heads and keys");
  pkv::ChunkArgs a = {};
  a.out = out;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.q_offsets = q_offsets;
  a.part = static_cast<float*>(workspace);
  a.cuts = reinterpret_cast<pkv::ChunkCut*>(static_cast<uint8_t*>(workspace) + chunk_partials(d));
  a.c2 = std::max(std::fabs(scale) * 1.4426950408889634f, std::numeric_limits<float>::denorm_min());
  a.negate = scale < 0.f;
  a.grid = device_sms();
  a.num_tokens = num_tokens;
  a.num_seqs = d->num_seqs;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.group = d->num_q_heads / d->num_kv_heads;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_blocks = d->num_blocks;
  a.tile_tokens = 128 / a.group;
  // At most so many units, from the host's view of the lengths.
  const int64_t units = (static_cast<int64_t>(num_tokens) / (2 * a.tile_tokens) + d->num_seqs) * d->num_kv_heads;
  a.whole_units = units > a.grid ? 0 : static_cast<int64_t>(a.max_blocks) * pkv::kBlockSize <= pkv::kWholeKeys ? 2 : 1;
  CUtensorMap mq, mk, mv;
  if ((rc = make_query_map(&mq, q, num_tokens, d, a.group)) != PKV_OK) return rc;
  if ((rc = make_block_map(&mk, k_cache, d)) != PKV_OK) return rc;
  if ((rc = make_block_map(&mv, v_cache, d)) != PKV_OK) return rc;
  cudaError_t e = cudaSuccess;
  with_type_and_dim(d, [&](auto t, auto dim) {
    using T = decltype(t);
    constexpr int D = decltype(dim)::value;
    constexpr auto kern = pkv::chunk_attention_kernel<T, D>;
    e = configure_smem<kern>(pkv::ChunkShape<D>::kSmem);
    if (e == cudaSuccess)
      e = launch(kern, dim3(a.grid), 1, pkv::kChunkThreads, pkv::ChunkShape<D>::kSmem, stream, mq, mk, mv, a);
    if (e == cudaSuccess && a.grid > 1 && a.whole_units != 2)
      e = launch(pkv::merge_chunk_kernel<T, D>, dim3(a.grid - 1, pkv::kChunkRows / pkv::kChunkMergeRows), 1,
                 pkv::kChunkMergeThreads, 0, stream, a);
  });
  if (e != cudaSuccess) return cuda_fail(e, "chunk_attention_kernel launch");
  return PKV_OK;
}

// ------------------------------------------------------------------ block-sparse decode

int update_bounds_impl(const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* q_offsets, int32_t num_tokens, int8_t* bounds, float* scales, const pkv_dims* d,
                       cudaStream_t stream) {
  int rc = check_dims(d, false);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return pkv_fail(PKV_ERR_INVALID_ARG, "update_bounds: num_tokens < 0");
  if (d->num_seqs == 0 || (q_offsets && num_tokens == 0)) return PKV_OK;
  if ((rc = check_tables(d, block_tables, context_lens, "update_bounds")) != PKV_OK) return rc;
  if (!k_cache || !bounds || !scales) return pkv_fail(PKV_ERR_INVALID_ARG, "update_bounds: NULL pointer");
  if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(scales, 4) || !aligned(q_offsets, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, "update_bounds: misaligned pointer (cache and bounds need 16 bytes)");
  pkv::BoundArgs a = {k_cache,      block_tables,        context_lens,  q_offsets, bounds, scales, d->num_seqs, d->num_kv_heads,
                      d->num_blocks, d->max_blocks_per_seq, num_tokens, 0};
  // Where sequence b's items start, plus what the last can have (beside the kernel).
  a.num_items = q_offsets ? static_cast<int64_t>(num_tokens) / pkv::kBlockSize + 2 * static_cast<int64_t>(d->num_seqs)
                          : d->num_seqs;
  const int64_t grid = (a.num_items * d->num_kv_heads + pkv::kBoundWarps - 1) / pkv::kBoundWarps;
  if (grid > INT_MAX) return pkv_fail(PKV_ERR_UNSUPPORTED, "update_bounds: too many blocks");
  cudaError_t e = cudaSuccess;
  with_type_and_dim(d, [&](auto t, auto dim) {
    e = launch(pkv::update_bounds_kernel<decltype(t), decltype(dim)::value>, dim3(static_cast<unsigned>(grid)), 1,
               pkv::kBoundWarps * 32, 0, stream, a);
  });
  if (e != cudaSuccess) return cuda_fail(e, "update_bounds_kernel launch");
  return PKV_OK;
}

// Scores and choice in one launch, without a workspace: tables of at most kWholeThreads
// blocks, as many (sequence, KV head) pairs as CTAs are on the SMs at once.  Up to 256
// blocks each, 8 KV heads: 32 sequences 7.5 us against 9.2 with two launches, 64 13.1
// against 11.9 (its CTAs are twice as large and wait for their rows as a whole), 256 45
// against 37.  With 5 sequences the binding's time counts, 27 us against 36 with the
// attention after it.
bool select_whole(const pkv_dims* d) {
  return d->max_blocks_per_seq <= pkv::kWholeThreads &&
         static_cast<int64_t>(d->num_seqs) * d->num_kv_heads <= pkv::kWholeUnits;
}

size_t select_workspace(const pkv_dims* d) {
  if (select_whole(d)) return 0;
  return align256(static_cast<size_t>(d->num_seqs) * d->num_kv_heads * d->max_blocks_per_seq * sizeof(uint32_t));
}

int select_blocks_impl(const pkv::SelectArgs& args, void* workspace, size_t workspace_bytes, const pkv_dims* d,
                       cudaStream_t stream) {
  int rc = check_dims(d, true);
  if (rc != PKV_OK) return rc;
  pkv::SelectArgs a = args;
  if (a.num_selected < 1 || a.sink < 0 || a.recent < 1)
    return pkv_fail(PKV_ERR_INVALID_ARG, "select_blocks: num_selected and recent_blocks from 1, sink_blocks from 0");
  if (static_cast<int64_t>(a.sink) + a.recent > a.num_selected)
    return pkv_fail(PKV_ERR_INVALID_ARG, "select_blocks: more blocks always kept than selected");
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "select_blocks: at most 65535 sequences and KV heads");
  if (d->num_seqs == 0) return PKV_OK;
  if ((rc = check_tables(d, a.block_tables, a.context_lens, "select_blocks")) != PKV_OK) return rc;
  if (!a.q || !a.bounds || !a.scales || !a.selected) return pkv_fail(PKV_ERR_INVALID_ARG, "select_blocks: NULL pointer");
  if (!aligned(a.q, 16) || !aligned(a.bounds, 16) || !aligned(a.scales, 4) || !aligned(a.selected, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, "select_blocks: misaligned pointer (q and bounds need 16 bytes)");
  const bool scored = d->max_blocks_per_seq > a.num_selected;  // else every block is chosen
  const size_t need = scored ? select_workspace(d) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return pkv_fail(PKV_ERR_INVALID_ARG, "select_blocks: workspace missing, too small (" + std::to_string(need) +
                                             " bytes needed) or not 256-byte aligned");
  a.keys = static_cast<uint32_t*>(workspace);
  a.num_seqs = d->num_seqs;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.group = d->num_q_heads / d->num_kv_heads;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  cudaError_t e = cudaSuccess;
  const bool whole = scored && select_whole(d);
  if (scored) {
    const int threads = whole ? pkv::kWholeThreads : pkv::kScoreThreads;
    // The CTAs of a table take its ranges of blocks in turn, a stride apart: one CTA for
    // each, but no more than about kScoreCtas in the grid, as those behind a context's
    // end cost time (32 sequences of 2,000 blocks in tables of 8,192, 8 KV heads: 40 us of
    // 16,384 CTAs, 27 of 4,096).  A CTA of several ranges makes its codes once: 128 full tables
    // of 2,048, group of 8, 140 us against 152; with 2,432 CTAs 145, 1,216 148, and where
    // lengths differ they leave SMs idle (101, 108, 125).
    const int64_t pairs = static_cast<int64_t>(d->num_kv_heads) * d->num_seqs;
    const int64_t ranges = std::min<int64_t>((a.max_blocks + threads - 1) / threads,
                                             std::max<int64_t>(1, pkv::kScoreCtas / pairs));
    const dim3 grid(static_cast<unsigned>(ranges * d->num_kv_heads), d->num_seqs);
    with_type_and_dim(d, [&](auto t, auto dim) {
      using T = decltype(t);
      constexpr int D = decltype(dim)::value;
      auto launch_group = [&](auto group) {
        constexpr int G = decltype(group)::value;
        const int smem = threads * 2 * D;
        if (whole) {
          e = configure_smem<pkv::score_blocks_kernel<T, D, G, true>>(smem);
          if (e == cudaSuccess)
            e = launch(pkv::score_blocks_kernel<T, D, G, true>, grid, 1, threads, smem, stream, a);
        } else {
          e = launch(pkv::score_blocks_kernel<T, D, G, false>, grid, 1, threads, smem, stream, a);
        }
      };
      if (a.group == 1)
        launch_group(std::integral_constant<int, 1>{});
      else if (a.group == 2)
        launch_group(std::integral_constant<int, 2>{});
      else if (a.group <= 4)
        launch_group(std::integral_constant<int, 4>{});
      else
        launch_group(std::integral_constant<int, 8>{});
    });
    if (e != cudaSuccess) return cuda_fail(e, "score_blocks_kernel launch");
  }
  if (whole) return PKV_OK;
  const dim3 grid(d->num_kv_heads, d->num_seqs);
  if (!scored || a.max_blocks <= 256 * pkv::kSelectRun) {
    e = launch(pkv::select_blocks_kernel<256>, grid, 1, 256, 0, stream, a);
  } else {
    const int most = pkv::select_place(pkv::kSelectCached) * 4 + 4;
    e = configure_smem<pkv::select_blocks_kernel<pkv::kSelectThreads>>(most);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(select_blocks_kernel)");
    const size_t smem = a.max_blocks <= pkv::kSelectThreads * pkv::kSelectRun
                            ? 0 : pkv::select_place(std::min(a.max_blocks, pkv::kSelectCached)) * 4 + 4;
    e = launch(pkv::select_blocks_kernel<pkv::kSelectThreads>, grid, 1, pkv::kSelectThreads, smem, stream, a);
  }
  if (e != cudaSuccess) return cuda_fail(e, "select_blocks_kernel launch");
  return PKV_OK;
}

int decode_sparse_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                       const int32_t* context_lens, const int32_t* selected, int32_t num_selected, float scale,
                       void* out, const pkv_dims* d, cudaStream_t stream) {
  int rc = check_dims(d, true);
  if (rc != PKV_OK) return rc;
  if (num_selected < 0) return pkv_fail(PKV_ERR_INVALID_ARG, "decode_attention_sparse: num_selected < 0");
  if (!std::isfinite(scale)) return pkv_fail(PKV_ERR_INVALID_ARG, "decode_attention_sparse: scale is not finite");
  if (d->num_seqs > 65535 || d->num_kv_heads > 65535)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "decode_attention_sparse: at most 65535 sequences and KV heads");
  if (d->num_seqs == 0) return PKV_OK;
  if ((rc = check_tables(d, block_tables, context_lens, "decode_attention_sparse")) != PKV_OK) return rc;
  if (!q || !k_cache || !v_cache || !out || (!selected && num_selected > 0))
    return pkv_fail(PKV_ERR_INVALID_ARG, "decode_attention_sparse: NULL pointer");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(selected, 4))
    return pkv_fail(PKV_ERR_INVALID_ARG, "decode_attention_sparse: misaligned pointer (q/out/caches need 16 bytes)");
  CUtensorMap mk, mv;
  if ((rc = g_maps.get(k_cache, d, false, &mk)) != PKV_OK) return rc;
  if ((rc = g_maps.get(v_cache, d, false, &mv)) != PKV_OK) return rc;
  pkv::DecodeArgs a = {};
  a.q = q;
  a.out = out;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.num_seqs = d->num_seqs;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.group = d->num_q_heads / d->num_kv_heads;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_blocks = d->num_blocks;
  // CTAs of a cluster: as many as are on the SMs at once, two on each, as long as every
  // warp has two blocks.  (One more doubling, two rounds of CTAs: 32 sequences x 8 heads
  // 80 us instead of 78 with the selection.)
  const int64_t units = static_cast<int64_t>(d->num_seqs) * d->num_kv_heads;
  unsigned cluster = 1;
  while (cluster < pkv::kMaxSparseCluster && units * cluster * 2 <= 2 * static_cast<int64_t>(device_sms()) &&
         static_cast<int64_t>(num_selected) >= 2 * static_cast<int64_t>(cluster) * 2 * pkv::kSparseWarps)
    cluster *= 2;
  cudaError_t e = cudaSuccess;
  with_type_and_dim(d, [&](auto t, auto dim) {
    constexpr int D = decltype(dim)::value;
    constexpr auto kern = pkv::decode_sparse_kernel<decltype(t), D>;
    e = configure_smem<kern>(pkv::SparseShape<D>::kSmem, true);
    if (e == cudaSuccess)
      e = launch(kern, dim3(cluster, d->num_kv_heads, d->num_seqs), cluster, pkv::kSparseWarps * 32,
                 pkv::SparseShape<D>::kSmem, stream, mk, mv, a, selected, num_selected, static_cast<int32_t>(cluster));
  });
  if (e != cudaSuccess) return cuda_fail(e, "decode_sparse_kernel launch");
  return PKV_OK;
}

}  // namespace

int pkv_long_context_error_word(unsigned* word) {
  *word = 0;
  return g_launched[current_device()].load(std::memory_order_relaxed) ? take_error_word(word) : cudaSuccess;
}

extern "C" {

int paged_kv_rope_init(pkv_rope* rope, const double* inv_freq, int32_t num_freqs, const int32_t* axes, int32_t num_axes,
                       int32_t interleaved, double factor) {
  if (!rope || !inv_freq) return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: NULL pointer");
  if (num_freqs < 8 || num_freqs > pkv::kMaxFreqs || num_freqs % 8 != 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: 8 to 64 frequencies, a multiple of 8");
  if (num_axes < 1 || num_axes > 4) return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: 1 to 4 position axes");
  if (!(std::fabs(factor) <= std::numeric_limits<float>::max()))
    return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: factor is not finite in float32");
  pkv_rope r = {};
  r.rot_dim = 2 * num_freqs;
  r.num_axes = num_axes;
  r.interleaved = interleaved != 0;
  r.factor = static_cast<float>(factor);
  for (int f = 0; f < num_freqs; ++f) {
    if (!std::isfinite(inv_freq[f])) return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: a frequency is not finite");
    const int axis = axes ? axes[f] : 0;
    if (axis < 0 || axis >= num_axes) return pkv_fail(PKV_ERR_INVALID_ARG, "rope_init: an axis is not among num_axes");
    r.axis_bits[f >> 5] |= static_cast<uint64_t>(axis) << (2 * (f & 31));
    // The fraction of the magnitude, below 1, so that the conversion is defined; a negative
    // frequency is its negative modulo 2^64.
    const double turns = std::fabs(inv_freq[f]) * 0.15915494309189533577;  // 1 / (2 pi)
    const uint64_t fraction = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
    r.turns[f] = inv_freq[f] < 0 ? 0 - fraction : fraction;
  }
  *rope = r;
  return PKV_OK;
}

int paged_kv_rope(const void* q, const void* k, const int32_t* positions, int32_t num_tokens, const pkv_rope* rope,
                  void* q_out, void* k_out, const pkv_rope_strides* strides, const pkv_dims* dims, void* stream) {
  return rope_impl(q, k, nullptr, positions, nullptr, num_tokens, rope, q_out, k_out, nullptr, nullptr, nullptr, strides,
                   dims, pkv::kRopeRows, "rope", static_cast<cudaStream_t>(stream));
}

int paged_kv_append_rope(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                         const int32_t* slot_mapping, int32_t num_tokens, const pkv_rope* rope, void* q_out,
                         void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                         const pkv_rope_strides* strides, const pkv_dims* dims, void* stream) {
  if (!k_scale != !v_scale) return pkv_fail(PKV_ERR_INVALID_ARG, "append_rope: give both k_scale and v_scale, or neither");
  return rope_impl(q, k_new, v_new, positions, slot_mapping, num_tokens, rope, q_out, k_cache, v_cache, k_scale, v_scale,
                   strides, dims, k_scale ? pkv::kRopePoolE4M3 : pkv::kRopePool16, "append_rope",
                   static_cast<cudaStream_t>(stream));
}

int paged_kv_update_bounds(const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                           const int32_t* q_offsets, int32_t num_tokens, int8_t* bounds, float* scales,
                           const pkv_dims* dims, void* stream) {
  return update_bounds_impl(k_cache, block_tables, context_lens, q_offsets, num_tokens, bounds, scales, dims,
                            static_cast<cudaStream_t>(stream));
}

int paged_chunk_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                          const int32_t* context_lens, const int32_t* q_offsets, int32_t num_tokens, float scale,
                          void* out, void* workspace, size_t workspace_bytes, const pkv_dims* dims, void* stream) {
  return chunk_attention_impl(q, k_cache, v_cache, block_tables, context_lens, q_offsets, num_tokens, scale, out,
                              workspace, workspace_bytes, dims, static_cast<cudaStream_t>(stream));
}

size_t paged_chunk_workspace_bytes(const pkv_dims* dims) {
  return check_dims(dims, true) == PKV_OK ? chunk_workspace(dims) : 0;
}

size_t paged_select_workspace_bytes(const pkv_dims* dims) {
  return check_dims(dims, true) == PKV_OK ? select_workspace(dims) : 0;
}

int paged_select_blocks(const void* q, const int8_t* bounds, const float* scales, const int32_t* block_tables,
                        const int32_t* context_lens, int32_t num_selected, int32_t sink_blocks, int32_t recent_blocks,
                        int32_t* selected, void* workspace, size_t workspace_bytes, const pkv_dims* dims, void* stream) {
  pkv::SelectArgs a = {};
  a.q = q;
  a.bounds = bounds;
  a.scales = scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.selected = selected;
  a.num_selected = num_selected;
  a.sink = sink_blocks;
  a.recent = recent_blocks;
  return select_blocks_impl(a, workspace, workspace_bytes, dims, static_cast<cudaStream_t>(stream));
}

int paged_decode_attention_sparse(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* selected, int32_t num_selected, float scale,
                                  void* out, const pkv_dims* dims, void* stream) {
  return decode_sparse_impl(q, k_cache, v_cache, block_tables, context_lens, selected, num_selected, scale, out, dims,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
