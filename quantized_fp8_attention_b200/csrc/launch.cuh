// launch.cuh -- launches that overlap with the end of the one before them.
#pragma once

namespace fqa {

// A launch that may begin while the kernel before it in the stream still runs
// (launch_overlapped() in fqa.cu): grid_wait() returns once that kernel has ended
// and its writes are visible, so it comes before the first access to global
// memory.  The accesses are plain loads: the kernel before may write what this
// one reads during this one's life, which the read-only path (__ldg) rules out,
// and a load of that kind may be moved above the wait.  grid_release() lets the
// next such launch begin once every CTA of this one has called it.  A kernel
// that takes tensor memory calls it after that: the next kernel's CTAs may take
// what is left, and wait for this kernel's end with it in hand.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace fqa
