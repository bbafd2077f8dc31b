// The rows of a batch in order of their adapter: a stable counting sort of M ids below L in one launch. Formulas and
// conventions: include/qgemm.h.
//
// A thread block for each adapter counts the ids below its own (its rows' first position) and its own ids, and then
// writes its rows in order, 4 ids a thread at a time, each after a prefix sum over the block. Every block reads all
// ids, 2 x 4 M bytes from L2; nothing is exchanged between blocks, and the order depends on the ids alone.
#include "serve.cuh"

namespace qg {
namespace {

__device__ __forceinline__ int4 ids_at(const int32_t* adapter, int i, int M) {
    if (i + 4 <= M) return load(reinterpret_cast<const int4*>(adapter + i));
    return make_int4(i < M ? load(adapter + i) : -1, i + 1 < M ? load(adapter + i + 1) : -1, i + 2 < M ? load(adapter + i + 2) : -1, -1);
}

__global__ void __launch_bounds__(1024) lora_group_kernel(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets) {
    __shared__ int2 part[32];
    __shared__ int held[2][32];
    const int l = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    grid_wait();
    grid_release();
    int less = 0, own = 0;
    for (int i = tid * 4; i < M; i += blockDim.x * 4) {
        const int4 v = ids_at(adapter, i, M);
        // ids below 0 are none: as whole numbers without sign they are above every adapter
        less += ((uint32_t)v.x < (uint32_t)l) + ((uint32_t)v.y < (uint32_t)l) + ((uint32_t)v.z < (uint32_t)l) + ((uint32_t)v.w < (uint32_t)l);
        own += (v.x == l) + (v.y == l) + (v.z == l) + (v.w == l);
    }
    less = __reduce_add_sync(0xffffffffu, less);
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) part[warp] = make_int2(less, own);
    __syncthreads();
    less = own = 0;
    for (int w = 0; w < warps; ++w) {
        less += part[w].x;
        own += part[w].y;
    }
    if (tid == 0) offsets[l] = less;
    if (l == L - 1) {
        if (tid == 0) offsets[L] = less + own;
        for (int i = less + own + tid; i < M; i += blockDim.x) row[i] = -1;
    }
    if (own == 0) return;
    int at = less;
    for (int i0 = 0, turn = 0; i0 < M; i0 += blockDim.x * 4, turn ^= 1) {
        const int i = i0 + tid * 4;
        const int4 v = i < M ? ids_at(adapter, i, M) : make_int4(-1, -1, -1, -1);
        const int n = (v.x == l) + (v.y == l) + (v.z == l) + (v.w == l);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31) held[turn][warp] = before;      // two turns' sums, so that one barrier each is enough
        __syncthreads();
        int to = at + before - n;
        for (int w = 0; w < warps; ++w) {
            const int s = held[turn][w];
            to += w < warp ? s : 0;
            at += s;
        }
        if (v.x == l) row[to++] = i;
        if (v.y == l) row[to++] = i + 1;
        if (v.z == l) row[to++] = i + 2;
        if (v.w == l) row[to++] = i + 3;
    }
}

}  // namespace

cudaError_t launch_lora_group(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets, cudaStream_t s) {
    const int threads = M >= 4096 ? 1024 : ((M + 3) / 4 + 31) / 32 * 32;
    return launch_behind(lora_group_kernel, dim3((unsigned)L), dim3(threads > 32 ? threads : 32), 0, 1, s, M, L, adapter, row, offsets);
}

}  // namespace qg
