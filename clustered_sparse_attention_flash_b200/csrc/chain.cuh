// Launching a kernel before the one ahead of it in the stream has ended
// (programmatic dependent launch), so that its launch and prologue hide behind
// that kernel's tail.  A kernel launched by launch_chained calls wait_previous()
// before it touches memory that another kernel may write or read, and reads such
// memory with coherent loads only: a non-coherent one (__ldg, __restrict__) is for
// memory that nothing writes while the kernel lives.  A kernel that calls
// launch_next() lets such a successor begin once all its own blocks have begun.
// Any other successor waits for its end as ever.
//
// The quantisation calls launch_next(); the product and the dequantisation are
// launched chained: 1.0 to 1.6 us less for quantisation and product (us, tokens x
// features x K, before / after: 1 x 2,048 x 2,048 6.9 / 5.9; 1 x 30,720 x 5,120
// 19.8 / 18.9; 128 x 5,120 x 5,120 17.0 / 15.5).  Kernels that fill every SM for
// long lose by it, since their early blocks spread unevenly (the product of 64
// tokens with 15,360 features after itself 15.0 / 19.2 us, a norm of 4,999 rows
// after itself 34.6 / 38.9): they do not call it.
#pragma once
#include <cuda_runtime.h>

namespace svg {

__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Returns when the kernels ahead have ended and their writes are visible.  The
// pointers pass through it, so that no load from them can move above it.
template <typename... P>
__device__ __forceinline__ void wait_previous(P*&... ptr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto pass = [](auto*& q) { asm volatile("" : "+l"(q)::"memory"); };
  (pass(ptr), ...);
}

// cluster 0: as the kernel itself says.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), int grid, int block, size_t smem, int cluster, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace svg
