// launch_order.cuh -- a kernel's place behind the work before it in its stream,
// for kernels launched so that they may begin while that work ends.
#pragma once

namespace jssm {

// Everything enqueued before this kernel has completed and its writes are
// visible.  Before any access to global memory.
__device__ __forceinline__ void after_earlier_work() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The next kernel of the stream may begin (it waits as above before it touches
// memory).
__device__ __forceinline__ void let_next_begin() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace jssm
