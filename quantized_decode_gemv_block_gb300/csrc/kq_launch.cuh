// Launch helpers shared by the paged-cache kernels (sm_103a).
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <string>

namespace kq {

// Waits until the kernels before this one on the stream have finished and their writes are
// visible. Every kernel launched by launch_pdl calls it before its first access to memory
// that another kernel may write or read.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream start its prologue.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The devices on which a kernel was allowed its dynamic shared memory (one of these per kernel, static).
struct SmemAllowed {
  std::atomic<unsigned long long> devices{0};
};
// Allows `kernel` dynamic shared memory up to `most` bytes: what the largest call of it takes, never a call's own
// figure. The attribute is the function's on its device, for all host threads, and a kernel needs it from 48 KB of
// static and dynamic memory together on.
template <typename Params>
int allow_smem(SmemAllowed& allowed, void (*kernel)(const Params), size_t most, const char* what, std::string* err) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev > 63 || !(allowed.devices.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess && dev < 64) allowed.devices.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) return 0;
  *err = std::string(what) + " shared memory: " + cudaGetErrorString(e);
  return -1;
}

// Launch as a programmatic dependent of the previous kernel on the stream: the grid may be placed
// while that kernel drains, and waits for it in grid_dependency_wait(). A kernel whose largest call passes 48 KB of
// shared memory is allowed it by allow_smem first.
template <typename Params>
int launch_pdl(void (*kernel)(const Params), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Params& p,
               const char* what, std::string* err) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) {
    *err = std::string(what) + " launch: " + cudaGetErrorString(e);
    return -1;
  }
  return 0;
}

}  // namespace kq
