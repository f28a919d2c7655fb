// Device helpers of the block-scaled cache's kernels: divisions by page and block,
// programmatic dependent launches, waits and elections of the tcgen05 kernel.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "block_params.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace vae4 {

// key / n for n a multiple of 16 up to 65536 and key < 2^30, m = ceil(2^38 /
// (n / 16)): with x = key / 16 < 2^26, x m < 2^64, and the excess of x m / 2^38
// over x / (n / 16) is below x / 2^38 < 2^-12 <= 1 / (n / 16).
__device__ __forceinline__ int div16(int key, unsigned long long m) {
  return (int)((unsigned long long)(unsigned)(key >> 4) * m >> 38);
}

// Programmatic dependent launch.  A kernel launched so may be placed while the
// one before it on the stream still runs: it touches global memory only after
// await_previous(), which every thread calls and which returns when that kernel
// has ended; the one after it may then be placed early in the same way (not
// before: it may read inputs, which earlier kernels wrote, ahead of its wait).
// What an earlier kernel may have written is read by load_dep, never through the
// read-only path (__ldg): that one is for data that nobody writes as long as the
// kernel is there, and a dependent is there while its inputs are being written.
__device__ __forceinline__ void await_previous() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
template <class T>
__device__ __forceinline__ T load_dep(const T *p) {
  return *p;
}
template <class P>
cudaError_t launch_dependent(void (*kernel)(P), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, const P &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

namespace tc {

// mbar_wait with everything but the first probe out of line: a kernel whose
// warps run many different loops is bound by instruction fetches, and a wait
// that is usually over should not take 40 instructions of each.
static __device__ __noinline__ bool mbar_wait_more(uint32_t bar, uint32_t parity,
                                                   volatile int *abort, long long limit) {
  return mbar_wait(bar, parity, abort, limit);
}
__device__ __forceinline__ bool mbar_wait_brief(uint32_t bar, uint32_t parity, volatile int *abort,
                                                long long limit) {
  if (limit >= kMinWaitLimit && mbar_try_wait(bar, parity)) return true;
  return mbar_wait_more(bar, parity, abort, limit);
}

// One lane of the (converged) warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r != 0;
}
}  // namespace tc
}  // namespace vae4
