// Kernel launches with a cluster size and, where `overlap` is set, as
// programmatic dependent launches: the kernel's blocks may start while the
// stream's previous kernel ends, and touch global memory only after
// griddepcontrol.wait.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
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

// Raises a kernel's limit of dynamic shared memory, once a device and thread: a
// table by the kernel's address, with room for all kernels of the library
// on eight devices. What finds no place is raised at every call.
inline cudaError_t allow_smem(const void* kern, size_t bytes) {
  struct Seen {
    const void* kern;
    int device;
  };
  constexpr uint32_t kPlaces = 1024, kTries = 64;
  static thread_local Seen seen[kPlaces];
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint32_t first = uint32_t((uint64_t(reinterpret_cast<uintptr_t>(kern)) >> 4) * 0x9E3779B1u >> 16) + uint32_t(device) * 97u;
  Seen* place = nullptr;
  for (uint32_t i = 0; i < kTries && place == nullptr; ++i) {
    Seen& s = seen[(first + i) % kPlaces];
    if (s.kern == kern && s.device == device) return cudaSuccess;
    if (s.kern == nullptr) place = &s;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess && place != nullptr) *place = {kern, device};
  return e;
}

}  // namespace mo
