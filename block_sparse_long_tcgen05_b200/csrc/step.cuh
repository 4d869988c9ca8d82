// What the serving kernels share: their ids in the device error word, and the order of kernels that
// follow one another in one call.
#pragma once
#include "ptx.cuh"

namespace msa {

// (ids 1 to 8: KernelId)
enum ServingKernelId : int {
  kKidRotate = 9,
  kKidPagedScan = 10,
  kKidPagedTopk = 11,
  kKidPagedAttn = 12,
  kKidPrefixScan = 13,
  kKidPagedSmall = 14,
};

// Kernels launched with programmatic stream serialisation. What the kernel before writes is read behind
// grid_wait, and by coherent loads: __ldg's path is for what stays as it is while a kernel runs, and this one
// runs beside its writer.
// Lets the next kernel's blocks start once every block of this one got here or ended.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits until the kernel before this one is done, its writes visible (and with it those that it waited for).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace msa
