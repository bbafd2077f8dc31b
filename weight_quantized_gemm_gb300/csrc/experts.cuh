// Device helpers shared by the 4-bit floating-point and mixture-of-experts kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace qg {

// Programmatic dependent launch: a kernel launched with the attribute may come up while the kernel
// before it in the stream still runs, once every block of that one has released it. grid_wait then
// waits until the earlier kernels are complete and their writes visible; nothing that they write, or
// read and this kernel writes, is touched before it. A kernel releases the next one only after its own
// wait: whatever comes up then knows every kernel but the one just before it to be complete, which the
// decode kernels rely on when they read a weight before they wait (QGEMM_OPT_LAUNCH_OVERLAP).
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What an earlier kernel may have written after this one came up is read with ordinary loads: the
// read-only path (__ldg) is for memory that nothing writes while the kernel lives.
template <class T>
__device__ __forceinline__ T load(const T* p) {
    return *p;
}
template <int DT>
__device__ __forceinline__ float load_as_float(const void* p, size_t i) {
    if constexpr (DT == DT_F32) return load(static_cast<const float*>(p) + i);
    else if constexpr (DT == DT_F16) return __half2float(load(static_cast<const __half*>(p) + i));
    else return __bfloat162float(load(static_cast<const __nv_bfloat16*>(p) + i));
}

}  // namespace qg
