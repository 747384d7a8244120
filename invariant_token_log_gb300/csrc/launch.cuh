// Launching a kernel that may start while its predecessor in the stream finishes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace {

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the previous kernel in the stream finishes (its launch latency hides
// behind that kernel's tail).  Only kernels that wait for their predecessor
// with griddep_wait() before touching global memory are launched this way:
// the forward's stream, cluster and merge kernels, the forward kernels of
// topk.cu, the norm's kernels and the 8-bit LM head.  (The logits path's
// backward is not: the wait made its element-by-element loads twice as slow.)
// cluster > 1: thread-block clusters of that many blocks along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), int64_t grid, int block, size_t smem, cudaStream_t stream,
                       int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  int n = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    n = 2;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace
