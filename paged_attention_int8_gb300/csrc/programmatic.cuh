// Programmatic launches: a kernel that starts while the one before it on the stream
// still runs, and waits inside for what it needs of it.
//
// Kernels of one call that work on disjoint data let the next start at once
// (launch_dependents at a block's start) and share the GPU.  The last block of each
// waits for the kernel before it ends, so that a kernel's end implies the end of all
// before it, which is what the call's last kernel waits for.  A call's first (or
// only) kernel is launched so too: every block of it waits for whatever ran before
// on the stream before it reads anything and before it lets the next kernel start,
// so that the launch and the set-up without inputs are all that overlaps (about 2 us
// of a call behind another).  The last kernel lets nothing start early: prefix blocks
// that came while a join still ran were spread unevenly over the SMs (48 us against
// 39 on 4 groups of 96 requests).
#pragma once

#include <cuda_runtime.h>

namespace paq8 {

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// In a block of the grid's last one: whichever way a thread leaves, it waits.
struct LastBlockWaits {
  bool last;
  __device__ ~LastBlockWaits() {
    if (last) wait_for_predecessor();
  }
};

// Launch attribute of a kernel that may start beside its predecessor.
struct BesidePredecessor {
  cudaLaunchAttribute attr[1];
  BesidePredecessor() {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
};

template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                          cudaStream_t stream, const A &...args) {
  BesidePredecessor b;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = b.attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace paq8
