// The rows of a batch in order of their adapter: a stable counting sort of M ids below L in one launch. Formulas and
// conventions: include/qgemm.h.
//
// A thread block for each adapter counts the ids below its own (its rows' first position) and its own ids, and then
// writes its rows in order. A thread takes 16 neighbouring ids, so that one prefix sum over the block orders 16384 of
// them, which are read once; a longer batch is read again for the second step. Every block reads all ids from L2;
// nothing is exchanged between blocks, and the order depends on the ids alone.
#include "serve.cuh"

namespace qg {
namespace {

constexpr int kIds = 16;        // of a thread at a time

// ids i .. i + 15; -1 past the end
__device__ __forceinline__ void fetch(const int32_t* adapter, int i, int M, int (&id)[kIds]) {
#pragma unroll
    for (int j = 0; j < kIds; j += 4) {
        int4 v = make_int4(-1, -1, -1, -1);
        if (i + j + 4 <= M) {
            v = load(reinterpret_cast<const int4*>(adapter + i + j));
        } else {
            if (i + j < M) v.x = load(adapter + i + j);
            if (i + j + 1 < M) v.y = load(adapter + i + j + 1);
            if (i + j + 2 < M) v.z = load(adapter + i + j + 2);
        }
        id[j] = v.x; id[j + 1] = v.y; id[j + 2] = v.z; id[j + 3] = v.w;
    }
}

__global__ void __launch_bounds__(1024) lora_group_kernel(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets) {
    __shared__ int s_less[32], s_own[2][32];
    const int l = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int turn = blockDim.x * kIds;
    grid_wait();
    grid_release();
    int id[kIds], less = 0, own = 0;
    for (int i0 = 0; i0 < M; i0 += turn) {      // (M <= 2^30: no overflow)
        fetch(adapter, i0 + tid * kIds, M, id);
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
            // ids below 0 are none: as whole numbers without sign they are above every adapter
            less += (uint32_t)id[j] < (uint32_t)l;
            own += id[j] == l;
        }
    }
    // Sums over the block in every thread: of all warps, and of the warps before this one.
    auto sums = [&](const int* part, int& before) {
        const int v = lane < warps ? part[lane] : 0;
        before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
        return __reduce_add_sync(0xffffffffu, v);
    };
    const int less_warp = __reduce_add_sync(0xffffffffu, less), own_warp = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) {
        s_less[warp] = less_warp;
        s_own[0][warp] = own_warp;
    }
    __syncthreads();
    int before;
    less = sums(s_less, before);
    const int all = sums(s_own[0], before);
    if (tid == 0) offsets[l] = less;
    if (l == L - 1) {
        if (tid == 0) offsets[L] = less + all;
        for (int i = less + all + tid; i < M; i += blockDim.x) row[i] = -1;
    }
    if (all == 0) return;
    int at = less;
    for (int i0 = 0, k = 0; i0 < M; i0 += turn, k ^= 1) {
        int n = own, here = all;
        if (M > turn) {             // the ids of this turn, and their counts
            fetch(adapter, i0 + tid * kIds, M, id);
            n = 0;
#pragma unroll
            for (int j = 0; j < kIds; ++j) n += id[j] == l;
            const int w = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) s_own[k ^ 1][warp] = w;      // two turns' sums, so that one barrier each is enough
            __syncthreads();
            here = sums(s_own[k ^ 1], before);
        }
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        int to = at + before + sum - n;
#pragma unroll
        for (int j = 0; j < kIds; ++j)
            if (id[j] == l) row[to++] = i0 + tid * kIds + j;
        at += here;
    }
}

}  // namespace

cudaError_t launch_lora_group(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets, cudaStream_t s) {
    const int threads = M >= 1024 * kIds ? 1024 : (M / kIds + 32) / 32 * 32;
    return launch_behind(lora_group_kernel, dim3((unsigned)L), dim3(threads), 0, 1, s, M, L, adapter, row, offsets);
}

}  // namespace qg
