// Device helpers shared by the kernels around the layers (adapters, norms, log probabilities).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.cuh"
#include "serve.h"

namespace qg {

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
// Barriers of the cluster's blocks, each thread arriving and waiting. The plain one orders lifetimes. With
// cluster_sync what any thread wrote to its own block's shared memory before is seen by all blocks after: its release
// is restricted to that memory, as one of all memory waits for the thread's loads in flight (a microsecond, where the
// next step's operands are on the way). cluster_sync_all also covers what was written to other blocks' shared memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    cluster_wait();
}
// Address of the same shared-memory variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t a) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// ---------------------------------------------------------------- eight values of a row
template <int DT>
struct Eight {
    static constexpr int kVecs = DT == DT_F32 ? 2 : 1;
    uint4 v[kVecs];
    // values i .. i + 7 of p (16-byte aligned)
    __device__ __forceinline__ void fetch(const void* p, size_t i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (DT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < kVecs; ++j) v[j] = load(q + j);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (DT == DT_F32) x[j] = __uint_as_float(w[j]);
            else if constexpr (DT == DT_BF16) x[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
            else x[j] = __half2float(__ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1)))));
        }
    }
    __device__ __forceinline__ void round_from(const float (&x)[8]) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int j = 0; j < 4 * kVecs; ++j) {
            if constexpr (DT == DT_F32) {
                w[j] = __float_as_uint(x[j]);
            } else if constexpr (DT == DT_F16) {
                const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    __device__ __forceinline__ void store(void* p, size_t i) const {
        uint4* q = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + i * (DT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < kVecs; ++j) q[j] = v[j];
    }
};

}  // namespace qg
