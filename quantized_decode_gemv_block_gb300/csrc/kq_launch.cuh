// Launch helpers shared by the paged-cache kernels (sm_103a).
#pragma once
#include <cuda_runtime.h>

#include <string>

namespace kq {

// Waits until the kernels before this one on the stream have finished and their writes are
// visible. Every kernel launched by launch_pdl calls it before its first access to memory
// that another kernel may write or read.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream start its prologue.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launch as a programmatic dependent of the previous kernel on the stream: the grid may be placed
// while that kernel drains, and waits for it in grid_dependency_wait().
template <typename Params>
int launch_pdl(void (*kernel)(const Params), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Params& p,
               const char* what, std::string* err, bool smem_is_allowed = false) {
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024 && !smem_is_allowed) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) {
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
    e = cudaLaunchKernelEx(&cfg, kernel, p);
  }
  if (e != cudaSuccess) {
    *err = std::string(what) + " launch: " + cudaGetErrorString(e);
    return -1;
  }
  return 0;
}

}  // namespace kq
