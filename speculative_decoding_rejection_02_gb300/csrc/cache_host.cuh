// What the host sides of the paged cache's calls share: the device's size, the status word,
// the launch, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/spec_cache.h"

namespace sv {

// The multiprocessors of the current device; 0 if it is not an sm_103.
inline int sm_count() {
  static int known[64];  // 0: not asked yet, -1: not an sm_103
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (known[dev] == 0) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    known[dev] = major == 10 && minor == 3 ? sms : -1;
  }
  return known[dev] > 0 ? known[dev] : 0;
}

// Where a call's status bits go on the current device, given the caller's word; NULL: no such
// place (spec_cache.cu).
__attribute__((visibility("hidden"))) unsigned* status_word(unsigned* given);

// Launch after the stream's earlier work, but with the launch itself prepared
// while that work still runs (the kernels begin with pdl_wait), in clusters of
// `cluster` blocks.
template <typename... A, typename... B>
int launch_cluster(void (*kernel)(A...), unsigned cluster, dim3 grid, int threads, size_t smem,
                   void* stream, const B&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return SPEC_OK;
  cudaGetLastError();
  return SPEC_ERR_CUDA;
}
template <typename... A, typename... B>
int launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, void* stream,
           const B&... args) {
  return launch_cluster(kernel, 1, grid, threads, smem, stream, args...);
}

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// A map of [x3][x2][x1][dim] 16-bit elements (strides in elements, not looked
// at for an extent of 1) for boxes of 64 elements x box1 x 1 x box3 in rows of
// 128 bytes, swizzled; elements past an extent read as zeros.
inline bool tensor_map(CUtensorMap* map, int dtype, const void* base, int dim, long long x1,
                long long s1, long long x2, long long s2, long long x3, long long s3,
                unsigned box1, unsigned box3) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return (Encode)fn;
  }();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)x1, (cuuint64_t)x2, (cuuint64_t)x3};
  const cuuint64_t least = ((cuuint64_t)dim * 2 + 15) / 16 * 16;
  const cuuint64_t strides[3] = {x1 > 1 ? (cuuint64_t)s1 * 2 : least,
                                 x2 > 1 ? (cuuint64_t)s2 * 2 : least,
                                 x3 > 1 ? (cuuint64_t)s3 * 2 : least};
  const cuuint32_t box[4] = {64, box1, 1, box3}, ones[4] = {1, 1, 1, 1};
  return encode(map, dtype == SPEC_CACHE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                4, const_cast<void*>(base), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sv
