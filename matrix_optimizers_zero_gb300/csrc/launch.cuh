// Kernel launches with a cluster size and, where `overlap` is set, as
// programmatic dependent launches: the kernel's blocks may start while the
// stream's previous kernel ends, and touch global memory only after
// griddepcontrol.wait.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace mo {

template <typename... Params, typename... Args>
inline cudaError_t launch_kernel(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, unsigned cluster, bool overlap,
                                 cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (overlap) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Raises a kernel's limit of dynamic shared memory, once a device.
inline cudaError_t allow_smem(const void* kern, size_t bytes) {
  struct Seen {
    const void* kern;
    int device;
  };
  static thread_local Seen seen[64];
  static thread_local int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < count; ++i)
    if (seen[i].kern == kern && seen[i].device == device) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess && count < 64) seen[count++] = {kern, device};
  return e;
}

}  // namespace mo
