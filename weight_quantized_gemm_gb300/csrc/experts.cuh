// Device helpers shared by the 4-bit floating-point and mixture-of-experts kernels.
#pragma once

namespace qg {

// Programmatic dependent launch: a kernel launched with the attribute may come up while the kernel
// before it in the stream still runs, once every block of that one has released it. grid_wait then
// waits until the earlier kernels are complete and their writes visible; nothing that they write, or
// read and this kernel writes, is touched before it.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace qg
