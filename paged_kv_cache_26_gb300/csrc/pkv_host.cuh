// Host pieces shared by the library's CUDA translation units: argument checks,
// TMA tensor maps of the pools, kernel attributes and dependent launches.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>
#include <string>
#include <type_traits>

#include "paged_kv.h"
#include "paged_kv_kernels.cuh"
#include "pkv_errors.h"

namespace {

constexpr int kMaxDevices = 64;

// The current device as an index below kMaxDevices (the last stands for those past it).
int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev < kMaxDevices ? dev : kMaxDevices - 1;
}

int device_sms() {
  static int sms[kMaxDevices] = {};
  const int dev = current_device();
  if (sms[dev] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    sms[dev] = v > 0 ? v : 1;
  }
  return sms[dev];
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int cuda_fail(cudaError_t e, const char* what) {
  return pkv_fail(PKV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_dims(const pkv_dims* d, bool need_q_heads) {
  if (!d) return pkv_fail(PKV_ERR_INVALID_ARG, "dims is NULL");
  if (d->num_seqs < 0 || d->num_kv_heads <= 0 || d->num_blocks <= 0 || d->max_blocks_per_seq < 0)
    return pkv_fail(PKV_ERR_INVALID_ARG, "dims: negative or zero size");
  if (d->dtype != PKV_DTYPE_FP16 && d->dtype != PKV_DTYPE_BF16)
    return pkv_fail(PKV_ERR_UNSUPPORTED, "dims: dtype must be fp16 or bf16");
  if (d->head_dim != 64 && d->head_dim != 128) return pkv_fail(PKV_ERR_UNSUPPORTED, "dims: head_dim must be 64 or 128");
  if (d->block_size != pkv::kBlockSize) return pkv_fail(PKV_ERR_UNSUPPORTED, "dims: block_size must be 16");
  if (static_cast<int64_t>(d->num_blocks) * d->num_kv_heads * pkv::kBlockSize >= (int64_t(1) << 31))
    return pkv_fail(PKV_ERR_UNSUPPORTED, "dims: num_blocks * num_kv_heads * 16 must be < 2^31");
  if (need_q_heads) {
    if (d->num_q_heads <= 0 || d->num_q_heads % d->num_kv_heads != 0)
      return pkv_fail(PKV_ERR_INVALID_ARG, "dims: num_kv_heads must divide num_q_heads");
    if (d->num_q_heads / d->num_kv_heads > 8)
      return pkv_fail(PKV_ERR_UNSUPPORTED, "dims: at most 8 query heads per KV head");
  }
  return PKV_OK;
}

// Reads and clears this translation unit's error word of the current device.
cudaError_t take_error_word(unsigned* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_pkv_error_word, sizeof(*word));
  if (e != cudaSuccess || *word == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_pkv_error_word, &zero, sizeof(zero));
}

// ------------------------------------------------------------------ tensor maps

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The pool as a 2-D tensor: rows = num_blocks * Hkv * 16 of head_dim elements;
// boxes of 16 rows x 128 bytes (64 fp16/bf16 elements or 128 E4M3 codes) with
// the 128-byte swizzle.
int make_cache_map(CUtensorMap* map, const void* cache, const pkv_dims* d, bool f8) {
  auto fn = encode_fn();
  if (!fn) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d->head_dim),
                              static_cast<cuuint64_t>(d->num_blocks) * d->num_kv_heads * pkv::kBlockSize};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d->head_dim) * (f8 ? 1 : 2)};
  const cuuint32_t box[2] = {f8 ? 128u : 64u, static_cast<cuuint32_t>(pkv::kBlockSize)};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType dt = f8                           ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : d->dtype == PKV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = fn(map, dt, 2, const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return pkv_fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(r) + ")");
  return PKV_OK;
}

// Small cache of encoded maps keyed by (address, shape, dtype): a decode loop
// reuses the same pool every step.
struct MapCache {
  struct Entry {
    const void* ptr = nullptr;
    int32_t nb = 0, hkv = 0, hd = 0, dt = -1;
    CUtensorMap map;
  };
  static constexpr int kEntries = 16;
  Entry e[kEntries];
  int next = 0;
  std::mutex mu;

  int get(const void* ptr, const pkv_dims* d, bool f8, CUtensorMap* out) {
    const int32_t dt = f8 ? -2 : d->dtype;
    std::lock_guard<std::mutex> lock(mu);
    for (auto& x : e)
      if (x.ptr == ptr && x.nb == d->num_blocks && x.hkv == d->num_kv_heads && x.hd == d->head_dim && x.dt == dt) {
        *out = x.map;
        return PKV_OK;
      }
    Entry& n = e[next];
    int rc = make_cache_map(&n.map, ptr, d, f8);
    if (rc != PKV_OK) return rc;
    n.ptr = ptr;
    n.nb = d->num_blocks;
    n.hkv = d->num_kv_heads;
    n.hd = d->head_dim;
    n.dt = dt;
    next = (next + 1) % kEntries;
    *out = n.map;
    return PKV_OK;
  }
};
MapCache g_maps;

// ------------------------------------------------------------------ launches

// Raise a kernel's dynamic shared-memory limit once per device (and ask for
// the largest shared-memory carveout).  The kernel is a template argument so
// that every kernel instantiation keeps its own flags.  wide_clusters: of more than
// eight CTAs.
template <auto kern>
cudaError_t configure_smem(int bytes, bool wide_clusters = false) {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < kMaxDevices && done[dev]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && wide_clusters) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
  return e;
}

// f(T, D) for the value type and head_dim of d.
template <typename F>
void with_type_and_dim(const pkv_dims* d, F&& f) {
  const bool bf16 = d->dtype == PKV_DTYPE_BF16;
  if (d->head_dim == 128)
    bf16 ? f(__nv_bfloat16{}, std::integral_constant<int, 128>{}) : f(__half{}, std::integral_constant<int, 128>{});
  else
    bf16 ? f(__nv_bfloat16{}, std::integral_constant<int, 64>{}) : f(__half{}, std::integral_constant<int, 64>{});
}

// A launch of `grid` CTAs in clusters of `cluster`, as a programmatic dependent
// launch: the kernel may start while the one before it in the stream finishes,
// and waits for it first (griddepcontrol.wait), so that what overlaps is the start.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, unsigned cluster, unsigned threads, size_t smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
