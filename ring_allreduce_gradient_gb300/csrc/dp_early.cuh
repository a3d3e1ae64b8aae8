// dp_early.cuh -- launches that overlap the end of the kernel before them: the
// CTAs come up while the last kernel of the stream drains.  Measured on calls
// in a row when these came, plain launches against these: the gradient norm of a 7 Mi-element
// list 9.3 -> 7.1 us, an 8-bit AdamW step of it 24.5 -> 21.8, decoding a
// 128x512 matrix (from a graph) 1.7 -> 1.3.
#pragma once

#include "dp_common.cuh"

namespace dpk {

// Comes first in such a kernel, before it touches global memory: everything
// before it in the stream has ended and is visible.  Global memory is read by
// plain loads: a read-only (.nc) load may be moved before the wait, and the
// kernel before may still be writing what it reads while this one exists.
__device__ __forceinline__ void wait_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What comes after this kernel may begin to set itself up once every CTA has
// come here or ended.  Called after wait_stream(), so that no more than one
// kernel's CTAs sit waiting beside those that run.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void stream_order() {
  wait_stream();
  let_next_start();
}

}  // namespace dpk

namespace dph {

template <typename P>
cudaError_t launch_early(void (*kernel)(P), const P& p, unsigned grid, unsigned threads,
                         cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace dph
