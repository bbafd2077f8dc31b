// The two ends of a mixture-of-experts layer: the router's choice of k experts for each token with
// the expert-sorted order of the chosen (token, expert) pairs, and the weighted sum of each token's
// expert output rows. Formulas and conventions: include/qgemm.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.cuh"
#include "experts.h"

namespace qg {
namespace {

// ---------------------------------------------------------------- routing
// A warp per token: lane i holds the logits of E / 32 neighbouring experts as order-preserving integer
// keys, and each of the k rounds takes the largest key by a warp reduction; of several lanes that
// hold it the lowest, and in it the lowest expert, is the lowest expert of all. A lane's keys are put
// in order first (up to 8 of them), so that taking one out of the warp is a shift and not another search
// through the lane's keys. A stable counting sort of the pairs by expert follows: each pair's rank among the
// block's pairs of its expert by warp matches, then the counts of the experts and blocks before, so the
// order depends on nothing but the input. A few tokens run in one thread block and one launch (128
// tokens of 128 experts there: 19 us against 8 in two launches); more run in two, where the second
// launch's blocks each sum the first's histograms themselves (at most kRouteBlocks x E counts, from
// L2) instead of waiting for a third launch that scans them. 8 tokens of 64 experts, top 8: 3.5 us (a
// launch and one pass of the chain above); 16384 tokens of 128, top 8: 18 us, where reading the logits
// takes 1.3. What bounds those is latency. Profiled by themselves on a cold cache the launches take 15.9 and
// 12.1 us. The first issues 470 warp instructions a token, 6 us if the issue slots were full; they are half
// busy, and warps wait for the block's barriers, for the rounds' chain of reduction, ballot and shuffle, and
// for their logits. The second fills 18 % of its issue slots and waits for the histograms.
constexpr int kSortWarps = 8;         // warps that rank a block's pairs
constexpr int kRouteThreads = 1024;
constexpr int kHeldPairs = 3584;      // experts of a block's pairs held in shared memory (more are read back)
static_assert((2 * 1024 + 1 + kSortWarps * 1024) * 4 + kHeldPairs * 2 <= 48 * 1024, "shared memory at 1024 experts");

struct RouteArgs {
    int T, E, k, renorm;
    const void* logits;
    long long ld;
    int32_t* expert;
    float* weight;
    int32_t* slot;
    int32_t* row;
    int32_t* offsets;
    int32_t* hist;      // [blocks][E]
    int per_block;      // tokens per block
};

// Keys grow with the value; 0 stands for an expert that cannot be chosen (-inf or NaN logit).
__device__ __forceinline__ uint32_t to_key(float x) {
    if (!(x > __uint_as_float(0xFF800000u))) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);   // -0 and 0 are one value
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// exp(x - top), where equal infinities count as equal values
__device__ __forceinline__ float rel_exp(float x, float top) { return x == top ? 1.f : expf(x - top); }

// Token t's choice by the calling warp: writes expert (also to held, from pair p0 on) and weight, and
// counts each expert's pairs.
template <int DT, int EL>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, int32_t* counts, int16_t* held, size_t p0) {
    constexpr bool kOrdered = EL <= 8;
    uint32_t key[EL], id[EL];
    const size_t from = (size_t)((long long)t * a.ld) + lane * EL;
#pragma unroll
    for (int j = 0; j < EL; ++j) {
        key[j] = lane * EL + j < a.E ? to_key(load_as_float<DT>(a.logits, from + j)) : 0u;
        id[j] = j;
    }
    uint32_t ids = 0, best = 0;      // kOrdered: the keys' places in the lane, 4 bits each
    if constexpr (kOrdered) {
        // exchanges of neighbours: equal keys keep their order
#pragma unroll
        for (int pass = 0; pass < EL; ++pass)
#pragma unroll
            for (int j = pass & 1; j + 1 < EL; j += 2) {
                const bool swap = key[j + 1] > key[j];
                const uint32_t hi = max(key[j], key[j + 1]), lo = min(key[j], key[j + 1]);
                const uint32_t i0 = swap ? id[j + 1] : id[j], i1 = swap ? id[j] : id[j + 1];
                key[j] = hi;
                key[j + 1] = lo;
                id[j] = i0;
                id[j + 1] = i1;
            }
#pragma unroll
        for (int j = 0; j < EL; ++j) ids |= id[j] << (4 * j);
        best = key[0];
    } else {
#pragma unroll
        for (int j = 0; j < EL; ++j) best = max(best, key[j]);
    }
    uint32_t first = 0, mine = 0;    // the largest key; lane r's: the r-th largest (0: none is left)
    int expert = -1;
    for (int r = 0; r < a.k; ++r) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0) break;
        if (r == 0) first = top;
        const int holder = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        int place;
        if constexpr (kOrdered) {
            place = (int)(ids & 15u);
        } else {
            place = 0;
#pragma unroll
            for (int j = EL - 1; j > 0; --j) place = key[j] == top ? j : place;
            if (key[0] == top) place = 0;
        }
        const int e = __shfl_sync(0xffffffffu, lane * EL + place, holder);
        if (lane == r) {
            mine = top;
            expert = e;
        }
        if (lane == holder) {
            if constexpr (kOrdered) {
#pragma unroll
                for (int j = 0; j + 1 < EL; ++j) key[j] = key[j + 1];
                key[EL - 1] = 0u;
                ids >>= 4;
                best = key[0];
            } else {
                best = 0;
#pragma unroll
                for (int j = 0; j < EL; ++j) {
                    if (j == place) key[j] = 0u;
                    best = max(best, key[j]);
                }
            }
        }
    }
    const float top = from_key(first), w = mine ? rel_exp(from_key(mine), top) : 0.f;
    float all = w;
    if (!a.renorm) {
        // over all experts: the ones not chosen are still in key, the chosen ones' terms are w
#pragma unroll
        for (int j = 0; j < EL; ++j)
            if (key[j]) all += rel_exp(from_key(key[j]), top);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane < a.k) {
        const size_t at = (size_t)t * a.k + lane;
        a.expert[at] = expert;
        a.weight[at] = mine ? w / all : 0.f;
        if (at - p0 < kHeldPairs) held[at - p0] = (int16_t)expert;
        if (expert >= 0) atomicAdd(counts + expert, 1);
    }
}

// The choice of tokens [t0, t1) by all warps of the block; counts[e] gets the block's pairs per
// expert (shared memory, cleared here; integer sums, so their order does not matter).
template <int DT, int EL>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int t0, int t1, int32_t* counts, int16_t* held) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) counts[e] = 0;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    for (int t = t0 + (int)(threadIdx.x >> 5); t < t1; t += warps)
        choose<DT, EL>(a, t, threadIdx.x & 31, counts, held, (size_t)t0 * a.k);
    __syncthreads();
}

// Stable positions of pairs [p0, p1) to slot: base[e] (none: 0) plus the pair's rank among the block's
// pairs of its expert; with base, the token to row, too. start: [kSortWarps][E] shared memory. Every
// thread of the block calls it.
__device__ __forceinline__ void place_block(const RouteArgs& a, int p0, int p1, const int16_t* held, const int32_t* base, int32_t* start) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * a.E; i += blockDim.x) start[i] = 0;
    __syncthreads();
    const int seg = ((p1 - p0 + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int b = min(p0 + warp * seg, p1), e1 = min(b + seg, p1), full = b + (e1 - b + 31) / 32 * 32;
    auto expert = [&](int p) { return p >= e1 ? -1 : (p - p0 < kHeldPairs ? (int)held[p - p0] : a.expert[p]); };
    if (warp < kSortWarps) {
        for (int p = b + lane; p < full; p += 32) {
            const int e = expert(p);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && lane == __ffs(same) - 1) start[warp * a.E + e] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int at = base ? base[e] : 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = start[w * a.E + e];
            start[w * a.E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    if (warp < kSortWarps) {
        for (int p = b + lane; p < full; p += 32) {
            const int e = expert(p);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            int at = -1;
            if (e >= 0) {
                at = start[warp * a.E + e] + __popc(same & ((1u << lane) - 1u));
                if (base) a.row[at] = p / a.k;
            }
            if (p < e1) a.slot[p] = at;
            __syncwarp();
            if (e >= 0 && lane == __ffs(same) - 1) start[warp * a.E + e] += __popc(same);
            __syncwarp();
        }
    }
}

// Exclusive prefix sum of v[0 .. E) into out[0 .. E], by the block's first warp.
__device__ __forceinline__ void prefix(const int32_t* v, int32_t* out, int E) {
    if (threadIdx.x < 32) {
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + threadIdx.x, x = e < E ? v[e] : 0;
            int s = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if ((int)threadIdx.x >= o) s += y;
            }
            if (e < E) out[e] = carry + s - x;
            carry += __shfl_sync(0xffffffffu, s, 31);
        }
        if (threadIdx.x == 0) out[E] = carry;
    }
    __syncthreads();
}

template <int DT, int EL>
__global__ void __launch_bounds__(kRouteThreads) route_small_kernel(const RouteArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int16_t held[kHeldPairs];
    grid_wait();
    grid_release();
    int32_t *counts = sm, *first = sm + a.E, *start = first + a.E + 1;
    choose_block<DT, EL>(a, 0, a.T, counts, held);
    prefix(counts, first, a.E);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = first[e];
    for (int p = first[a.E] + threadIdx.x; p < a.T * a.k; p += blockDim.x) a.row[p] = -1;
    place_block(a, 0, a.T * a.k, held, first, start);
}

template <int DT, int EL>
__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const RouteArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int16_t held[kHeldPairs];
    const int t0 = min(blockIdx.x * a.per_block, a.T), t1 = min(t0 + a.per_block, a.T);
    choose_block<DT, EL>(a, t0, t1, sm, held);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(size_t)blockIdx.x * a.E + e] = sm[e];
    place_block(a, t0 * a.k, t1 * a.k, held, nullptr, sm + a.E);
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const RouteArgs a) {
    extern __shared__ int32_t sm[];
    int32_t *total = sm, *before = sm + a.E, *first = before + a.E;
    grid_wait();
    for (int e = threadIdx.x; e < 2 * a.E; e += blockDim.x) sm[e] = 0;
    __syncthreads();
    // the pairs per expert in all blocks, and in the blocks before this one
    const int groups = max((int)blockDim.x / a.E, 1);
    for (int i = threadIdx.x; i < groups * a.E; i += blockDim.x) {
        const int g = i / a.E, e = i - g * a.E;
        int all = 0, mine = 0;
#pragma unroll 8
        for (int b = g; b < (int)gridDim.x; b += groups) {
            const int c = load(a.hist + (size_t)b * a.E + e);
            all += c;
            mine += b < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(total + e, all);
        atomicAdd(before + e, mine);
    }
    __syncthreads();
    prefix(total, first, a.E);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = first[e];
        for (int p = first[a.E] + threadIdx.x; p < a.T * a.k; p += blockDim.x) a.row[p] = -1;
    }
    const int t0 = min(blockIdx.x * a.per_block, a.T), p0 = t0 * a.k, p1 = min(t0 + a.per_block, a.T) * a.k;
    for (int p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
        const int e = load(a.expert + p);
        if (e < 0) continue;
        const int at = first[e] + before[e] + a.slot[p];
        a.slot[p] = at;
        a.row[at] = p / a.k;
    }
}

template <int DT, int EL>
cudaError_t route_el(RouteArgs a, cudaStream_t s) {
    const size_t sort = (size_t)kSortWarps * a.E * sizeof(int32_t);
    if (!route_needs_workspace(a.T)) {
        const int threads = 32 * (a.T > kSortWarps ? a.T : kSortWarps);     // a warp per token
        return launch_behind(route_small_kernel<DT, EL>, 1, threads, (2 * a.E + 1) * sizeof(int32_t) + sort, 1, s, a);
    }
    // blocks of at least 8 tokens, a warp per token up to 32 of them
    const int want = (a.T + 7) / 8;
    const int blocks = want < kRouteBlocks ? want : kRouteBlocks;
    a.per_block = (a.T + blocks - 1) / blocks;
    const int warps = a.per_block < kSortWarps ? kSortWarps : (a.per_block < kRouteThreads / 32 ? a.per_block : kRouteThreads / 32);
    // (the first launch neither comes up early nor lets the second: blocks that wait beside the ones that
    // choose made 1024 tokens 8.5 -> 11 us)
    route_choose_kernel<DT, EL><<<blocks, 32 * warps, a.E * sizeof(int32_t) + sort, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_behind(route_place_kernel, blocks, kRouteThreads, (3 * a.E + 1) * sizeof(int32_t), 1, s, a);
    return e;
}

template <int DT>
cudaError_t route_dt(const RouteArgs& a, cudaStream_t s) {
    if (a.E <= 32) return route_el<DT, 1>(a, s);
    if (a.E <= 64) return route_el<DT, 2>(a, s);
    if (a.E <= 128) return route_el<DT, 4>(a, s);
    if (a.E <= 256) return route_el<DT, 8>(a, s);
    if (a.E <= 512) return route_el<DT, 16>(a, s);
    return route_el<DT, 32>(a, s);
}

// ---------------------------------------------------------------- combining
// out[t] = sum_j weight[t][j] * Y[slot[t][j]] + residual[t], in float32, in the order of j, rounded
// once. HBM bounds it (k rows in, one out, each byte once); a thread takes 8 columns of one token and
// has up to four rows' loads in flight. 16384 tokens of 8 x 2560 in bf16: 111 us, 6.8 TB/s, the measured
// copy rate; 8 tokens of 4 x 4096: 1.6 us.
struct CombineArgs {
    int T, k, N, R;
    const void* Y;
    const int32_t* slot;
    const float* weight;
    const void* residual;
    void* out;
};

// 16 bytes at p, or zeros where there is nothing to read: a load under a predicate, so that the loads
// of several rows are in flight together (a branch for each instead: 138 us where this takes 111).
__device__ __forceinline__ uint4 load_if(bool in, const uint4* p) {
    uint4 r = make_uint4(0, 0, 0, 0);
    asm volatile("{\n.reg .pred in;\nsetp.ne.s32 in, %5, 0;\n@in ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w) : "l"(p), "r"((int)in));
    return r;
}

template <int DT, int V>
struct Vec {   // V consecutive values (V = 8: 16-byte loads; V = 1: any N)
    static constexpr int kVecs = V == 1 ? 1 : (DT == DT_F32 ? 2 : 1);
    uint4 raw[kVecs];
    __device__ __forceinline__ void fetch(const void* p, size_t i, bool in) {
        if constexpr (V == 1) {
            raw[0].x = in ? __float_as_uint(load_as_float<DT>(p, i)) : 0u;
        } else {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (DT == DT_F32 ? 4 : 2));
#pragma unroll
            for (int v = 0; v < kVecs; ++v) raw[v] = load_if(in, q + v);
        }
    }
    __device__ __forceinline__ void values(float (&x)[V]) const {
        if constexpr (V == 1) {
            x[0] = __uint_as_float(raw[0].x);
        } else {
            uint32_t w[4 * kVecs];
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                w[4 * v] = raw[v].x; w[4 * v + 1] = raw[v].y; w[4 * v + 2] = raw[v].z; w[4 * v + 3] = raw[v].w;
            }
#pragma unroll
            for (int c = 0; c < V; ++c) {
                if constexpr (DT == DT_F32) x[c] = __uint_as_float(w[c]);
                else if constexpr (DT == DT_F16) x[c] = __half2float(__ushort_as_half((unsigned short)(w[c >> 1] >> (16 * (c & 1)))));
                else x[c] = __uint_as_float((c & 1) ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
            }
        }
    }
};

template <int DT, int V>
__device__ __forceinline__ void store_vec(void* p, size_t i, const float* x) {
    if constexpr (V == 1) {
        if constexpr (DT == DT_F32) static_cast<float*>(p)[i] = x[0];
        else if constexpr (DT == DT_F16) static_cast<__half*>(p)[i] = __float2half_rn(x[0]);
        else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x[0]);
    } else if constexpr (DT == DT_F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if constexpr (DT == DT_F16) {
                const __half2 h = __floats2half2_rn(x[2 * c], x[2 * c + 1]);
                w[c] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * c], x[2 * c + 1]);
                w[c] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + i * 2) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// block (64, 4): 64 runs of V columns of 4 tokens
template <int DT, int ODT, int V>
__global__ void __launch_bounds__(256, DT == DT_F32 ? 4 : 6) combine_kernel(const CombineArgs a) {
    grid_wait();
    grid_release();
    const int t = blockIdx.x * 4 + threadIdx.y;
    const int n = (blockIdx.y * 64 + threadIdx.x) * V;
    if (t >= a.T || n >= a.N) return;
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
    // Four rows at a time; the next four's slots come while these rows do, so that each four wait for one
    // round trip.
    const int32_t* slot = a.slot + (size_t)t * a.k;
    const float* weight = a.weight + (size_t)t * a.k;
    int s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = j < a.k ? load(slot + j) : -1;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        Vec<DT, V> y[4];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = s[j] >= 0 && s[j] < a.R;    // a pair that was not placed adds nothing
            y[j].fetch(a.Y, (size_t)s[j] * a.N + n, in);
            w[j] = in ? load(weight + j0 + j) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = j0 + 4 + j < a.k ? load(slot + j0 + 4 + j) : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x[V];
            y[j].values(x);
#pragma unroll
            for (int c = 0; c < V; ++c) acc[c] = fmaf(w[j], x[c], acc[c]);
        }
    }
    if (a.residual) {
        Vec<ODT, V> r;
        r.fetch(a.residual, (size_t)t * a.N + n, true);
        float x[V];
        r.values(x);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] += x[c];
    }
    store_vec<ODT, V>(a.out, (size_t)t * a.N + n, acc);
}

template <int DT, int ODT>
cudaError_t combine_v(const CombineArgs& a, cudaStream_t s) {
    const int columns = a.N % 8 == 0 ? a.N / 8 : a.N;
    const dim3 grid((a.T + 3) / 4, (columns + 63) / 64), block(64, 4);
    return a.N % 8 == 0 ? launch_behind(combine_kernel<DT, ODT, 8>, grid, block, 0, 1, s, a)
                        : launch_behind(combine_kernel<DT, ODT, 1>, grid, block, 0, 1, s, a);
}
template <int DT>
cudaError_t combine_dt(const CombineArgs& a, int out_dtype, cudaStream_t s) {
    switch (out_dtype) {
        case DT_F32: return combine_v<DT, DT_F32>(a, s);
        case DT_F16: return combine_v<DT, DT_F16>(a, s);
        default: return combine_v<DT, DT_BF16>(a, s);
    }
}

}  // namespace

cudaError_t launch_moe_route(int T, int E, int k, const void* logits, int dtype, long long ld, int renorm, int32_t* expert,
                             float* weight, int32_t* slot, int32_t* row, int32_t* offsets, void* workspace, cudaStream_t s) {
    RouteArgs a{T, E, k, renorm, logits, ld, expert, weight, slot, row, offsets, static_cast<int32_t*>(workspace), 0};
    switch (dtype) {
        case DT_F32: return route_dt<DT_F32>(a, s);
        case DT_F16: return route_dt<DT_F16>(a, s);
        default: return route_dt<DT_BF16>(a, s);
    }
}

cudaError_t launch_moe_combine(int T, int k, int N, int R, const void* Y, int y_dtype, const int32_t* slot,
                               const float* weight, const void* residual, void* out, int out_dtype, cudaStream_t s) {
    const CombineArgs a{T, k, N, R, Y, slot, weight, residual, out};
    switch (y_dtype) {
        case DT_F32: return combine_dt<DT_F32>(a, out_dtype, s);
        case DT_F16: return combine_dt<DT_F16>(a, out_dtype, s);
        default: return combine_dt<DT_BF16>(a, out_dtype, s);
    }
}

}  // namespace qg
