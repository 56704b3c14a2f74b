// What the host sides of the paged cache's calls share: the device's size, the status word,
// the launch.
#pragma once
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

}  // namespace sv
