// Low-rank adapters beside a shared projection: Y[m] += scale_l B_l (A_l X[m]) for the rows of every adapter, in one
// launch. This file has the kernel for few rows, lora_many.cuh the one for many; instantiated for f16 and bf16 operands, each for
// rows of Y that start 16-byte aligned (lora_f16.cu, lora_bf16.cu) and for rows that need not (lora_loose_f16.cu, lora_loose_bf16.cu).
// In one kernel the second form's code made the first slower (8192 x 4096 x 14336 at rank 16 96 -> 98 us).
//
// A cluster of thread blocks takes up to 16 rows of one adapter. Its blocks share K in the first product (H = X A^T,
// R values a row), join their parts of H in distributed shared memory, each in the same order, and share N in the
// second one (H B^T), so neither product needs scratch memory or a second launch. What bounds it is a chain of round
// trips: the offsets, the first product's operands, the join, the second one's, the store. 16 rows of 16 adapters,
// 4096 x 4096 at rank 16: 4.6 us in a graph, in which the parts take some 1700 cycles (tile and rows), 1250 (the first
// product, one step a warp), 600 (its warps' sums), 700 (asking for B and Y), 1400 (the join) and 1500 (the second
// product). 77 rows of 24 adapters of ranks up to 64, 9728 x 2560, float32 Y: 13.9 us, of which the first product's five
// steps a warp take 4 (15 MB, most of which HBM needs 2.3 for).
//
// Both products run on 16x8x16 tensor-core steps from registers, without a copy through shared memory: the order of
// the summed index is free as long as both operands keep to it, so a lane takes 16 neighbouring bytes of a row as its
// values of two steps; and the order of the columns of the second product is chosen so that a lane ends with 8
// neighbouring values of Y's row.
//
// H is a float32 sum and enters the second product as a sum of 16-bit terms (hi = its nearest 16-bit value, then the
// nearest to what is left): three of bf16 for float32 Y, which hold it whole; two of bf16 for 16-bit Y, off by up to 2^-17 of
// it, where Y's own rounding is 2^-12 or 2^-9 (a third term is half as many products again, and its place in shared
// memory); two of f16, off by up to 2^-23 of it, as float32's rounding is 2^-24, or by 2^-39 of the row's largest H if that
// is more. f16 terms are of H scaled by a power of two for each row, so that they neither overflow nor lose their second
// term to f16's smallest exponent.
#pragma once

#include "serve.cuh"

namespace qg {
namespace lora {

constexpr int kThreads = 256, kWarps = 8;

struct Params {
    LoraArgs a;
};
// 16-bit terms that stand for a value of H
constexpr int terms_of(bool bf, int y_dtype) { return bf && y_dtype == DT_F32 ? 3 : 2; }

// 16 x 8 += 16 x 16 * 16 x 8
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// The 16-bit value nearest to x, as bits; x becomes what is left of it (0 where the value is infinite or NaN).
template <bool BF>
__device__ __forceinline__ uint32_t take_term(float& x) {
    float y;
    uint32_t bits;
    if constexpr (BF) {
        const __nv_bfloat16 h = __float2bfloat16_rn(x);
        bits = __bfloat16_as_ushort(h);
        y = __bfloat162float(h);
    } else {
        const __half h = __float2half_rn(x);
        bits = __half_as_ushort(h);
        y = __half2float(h);
    }
    x = fabsf(y) < __uint_as_float(0x7F800000u) ? x - y : 0.f;
    return bits;
}

// f16 terms are of H over a power of two that puts the row's largest finite |H| (its bits) between 2^14 and 2^15: half a step
// of the smallest f16 is then 2^-39 of it at most (with the largest between 1 and 2, an H of 2^-30 of it became 0, which
// counts where B's value for the largest is 0). This is that power.
__device__ __forceinline__ float row_unit(uint32_t top) { return __uint_as_float((max(top >> 23, 15u) - 14u) << 23); }
__device__ __forceinline__ float row_unit_inverse(uint32_t top) { return __uint_as_float((268u - max(top >> 23, 15u)) << 23); }
// |x|, and 0 where x is infinite or NaN: these need no unit, and must not set the others' (which were then beyond f16).
__device__ __forceinline__ float finite_size(float x) {
    x = fabsf(x);
    return x < __uint_as_float(0x7F800000u) ? x : 0.f;
}

// 4 values at h of all blocks, added in rank order, AT_ONCE of them asked for together: a round trip to another block takes
// some 700 cycles (16 rows, 16 adapters, with 8 together 4.5 us, with 4 4.8; of ranks up to 64 registers allow 4).
template <int AT_ONCE>
__device__ __forceinline__ float4 sum_of_blocks(const float* h, int blocks) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < blocks; k0 += AT_ONCE) {
        float4 o[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if (k0 + k < blocks) o[k] = ld_cluster_f32x4(in_block(h, k0 + k));
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if (k0 + k < blocks) {
                v.x += o[k].x; v.y += o[k].y; v.z += o[k].z; v.w += o[k].w;
            }
    }
    return v;
}
// H of all of K from the blocks' parts h: [rows][pitch], 16 * chunks columns, WIDTH pieces of 4 at a time; top: the bits
// of each row's largest finite |H| (f16; cleared before). Every thread of the block calls it.
template <bool BF, int WIDTH>
__device__ __forceinline__ void join_h(const float* h, float* sum, uint32_t* top, int pitch, int rows, int chunks, int blocks) {
    for (int c0 = 0; c0 < chunks * 4; c0 += WIDTH)
        for (int i = threadIdx.x; i < rows * WIDTH; i += kThreads) {
            const int row = i / WIDTH, c = c0 + i % WIDTH, at = row * pitch + c * 4;
            if (c >= chunks * 4) continue;
            float4 v;
            if (blocks == 1) v = *reinterpret_cast<const float4*>(h + at);
            else if (WIDTH <= 8 && blocks == 8) v = sum_of_blocks<8>(h + at, 8);
            else v = sum_of_blocks<4>(h + at, blocks);
            *reinterpret_cast<float4*>(sum + at) = v;
            if constexpr (!BF) {
                const float t = fmaxf(fmaxf(finite_size(v.x), finite_size(v.y)), fmaxf(finite_size(v.z), finite_size(v.w)));
                atomicMax(top + row, __float_as_uint(t));
            }
        }
}
// H's 16-bit terms, in the order in which the lanes take them: frag [chunks][terms][32]. Columns past the rank become
// zeros: A's zeros there times an infinite X were NaN.
template <bool BF, int TERMS>
__device__ __forceinline__ void make_terms(const float* sum, const uint32_t* top, uint4* frag, int pitch, int rank, int chunks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    for (int f = warp; f < chunks; f += kWarps) {
        float v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = g + 8 * i;
            const float4 o = *reinterpret_cast<const float4*>(sum + row * pitch + f * 16 + q * 4);
            const float by = BF ? 1.f : row_unit_inverse(top[row]);
            v[i][0] = o.x * by; v[i][1] = o.y * by; v[i][2] = o.z * by; v[i][3] = o.w * by;
        }
        if (f * 16 + 16 > rank)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (f * 16 + q * 4 + k >= rank) v[0][k] = v[1][k] = 0.f;
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
            uint32_t w[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = take_term<BF>(v[i][2 * k]), hi = take_term<BF>(v[i][2 * k + 1]);
                    w[i][k] = lo | hi << 16;
                }
            frag[(f * TERMS + t) * 32 + lane] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
        }
    }
}
// y[k] += scale * d[k] for the first `n` of 8 values, one at a time.
template <int YDT>
__device__ __forceinline__ void add_edge(void* y, const float (&d)[8], float scale, int n) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? load_as_float<YDT>(y, k) : 0.f;      // (all asked for before the first is stored)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= n) break;
        v[k] = fmaf(scale, d[k], v[k]);
        if constexpr (YDT == DT_F32) static_cast<float*>(y)[k] = v[k];
        else if constexpr (YDT == DT_F16) static_cast<__half*>(y)[k] = __float2half_rn(v[k]);
        else static_cast<__nv_bfloat16*>(y)[k] = __float2bfloat16_rn(v[k]);
    }
}

// Rows of Y that do not start 16-byte aligned: eight values of a row as the pairs n, n + 1, n + 8, n + 9, ... + 25, of which four
// neighbouring lanes have 32 columns without a gap. 77 rows of 24 adapters, ranks up to 64, beside 4096 x 5760 in bf16 take 14
// us aligned, 15 in rows of 5762 and 18 of 5761 values, 2000 rows of 100 adapters 28, 46 and 82 (with 8 neighbouring values a
// lane, one after the other, 40 and 280). Values past N are neither read nor written.
template <int YDT>
__device__ __forceinline__ void fetch_pairs(Eight<YDT>& y, const void* row, int n, int N) {
    uint32_t* w = reinterpret_cast<uint32_t*>(y.v);
    if constexpr (YDT == DT_F32) {
        const uint32_t* p = static_cast<const uint32_t*>(row);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n + 8 * t + i < N) w[2 * t + i] = load(p + n + 8 * t + i);
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(row);
        const bool words = (reinterpret_cast<uintptr_t>(p) & 2u) == 0;      // (n is even)
        uint16_t lo[4], hi[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = n + 8 * t;
            lo[t] = hi[t] = 0;
            if (words && c + 1 < N) {
                w[t] = load(reinterpret_cast<const uint32_t*>(p + c));
            } else {
                if (c < N) lo[t] = load(p + c);
                if (c + 1 < N) hi[t] = load(p + c + 1);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (!words || n + 8 * t + 1 >= N) w[t] = lo[t] | (uint32_t)hi[t] << 16;
    }
}
template <int YDT>
__device__ __forceinline__ void store_pairs(const Eight<YDT>& y, void* row, int n, int N) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(y.v);
    if constexpr (YDT == DT_F32) {
        uint32_t* p = static_cast<uint32_t*>(row);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n + 8 * t + i < N) p[n + 8 * t + i] = w[2 * t + i];
    } else {
        uint16_t* p = static_cast<uint16_t*>(row);
        const bool words = (reinterpret_cast<uintptr_t>(p) & 2u) == 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = n + 8 * t;
            if (words && c + 1 < N) {
                *reinterpret_cast<uint32_t*>(p + c) = w[t];
            } else {
                if (c < N) p[c] = (uint16_t)w[t];
                if (c + 1 < N) p[c + 1] = (uint16_t)(w[t] >> 16);
            }
        }
    }
}

// The q-th tile of `rows` rows over the adapters: its adapter, first position in `row`, and rows. Offsets are held to
// [0, M] and to the largest before them. Every thread of the block calls it.
//
// Up to 32 adapters each warp looks by itself; more are shared between the block's threads, neighbouring adapters a
// thread (96 rows of 1000 adapters, 4096 x 4096, 22 us; with 32 at a time in every warp 36).
struct TileSearch {
    int most[kWarps], tiles[kWarps], l, from, count;
};
__device__ __forceinline__ int max_up_to(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v = max(v, y);
    }
    return v;
}
__device__ __forceinline__ int sum_up_to(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += y;
    }
    return v;
}
__device__ __forceinline__ bool find_tile(const LoraArgs& a, int q, int rows, TileSearch& s, int& l, int& from, int& count) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = min(max(load(a.offsets), 0), a.M);
    if (a.L <= 32) {
        const int end = max(first, max_up_to(lane < a.L ? min(max(load(a.offsets + lane + 1), 0), a.M) : 0));
        int begin = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) begin = first;
        const int mine = (end - begin + rows - 1) / rows, sum = sum_up_to(mine);
        const uint32_t here = __ballot_sync(0xffffffffu, q < sum);
        if (!here) return false;
        l = __ffs(here) - 1;
        const int before = __shfl_sync(0xffffffffu, sum - mine, l), b = __shfl_sync(0xffffffffu, begin, l);
        const int e = __shfl_sync(0xffffffffu, end, l);
        from = b + (q - before) * rows;
        count = min(rows, e - from);
        return true;
    }
    constexpr int kEach = kMaxLoraAdapters / kThreads;
    const int each = (a.L + kThreads - 1) / kThreads, l0 = tid * each;
    int end[kEach], most = first;
#pragma unroll
    for (int j = 0; j < kEach; ++j) end[j] = j < each && l0 + j < a.L ? min(max(load(a.offsets + l0 + j + 1), 0), a.M) : 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) most = max(most, end[j]);
    const int up_to = max_up_to(most);
    if (lane == 31 && warp < kWarps) s.most[warp] = up_to;
    __syncthreads();
    int begin = __shfl_up_sync(0xffffffffu, up_to, 1);
    if (lane == 0) begin = first;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) begin = max(begin, s.most[w]);
    int mine = 0, at = begin;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        end[j] = max(end[j], at);
        mine += (end[j] - at + rows - 1) / rows;
        at = end[j];
    }
    int sum = sum_up_to(mine);
    if (lane == 31 && warp < kWarps) s.tiles[warp] = sum;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) sum += s.tiles[w];
        all += s.tiles[w];
    }
    if (q >= all) return false;
    int before = sum - mine;
    if (q >= before && q < sum) {
        at = begin;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int tiles = (end[j] - at + rows - 1) / rows;
            if (q >= before && q < before + tiles) {
                s.l = l0 + j;
                s.from = at + (q - before) * rows;
                s.count = min(rows, end[j] - s.from);
            }
            before += tiles;
            at = end[j];
        }
    }
    __syncthreads();
    l = s.l;
    from = s.from;
    count = s.count;
    return true;
}

// 16 or 8 bytes, zeros where `any` is not set: one instruction under a predicate, where a branch around each of a step's
// loads takes longer than the loads (77 rows of ranks up to 64: 15.4 -> 14.4 us).
__device__ __forceinline__ void load_if(uint4& v, const void* p, bool any) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)any));
}
__device__ __forceinline__ void load_if(uint2& v, const void* p, bool any) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t@p ld.global.v2.b32 {%0, %1}, [%2];\n\t}"
                 : "=&r"(v.x), "=&r"(v.y)
                 : "l"(p), "r"((int)any));
}

// Sixteen ranks at a time are a chunk; JT of them are in registers together.
template <int JT>
struct Shape {
    static constexpr int kRows = 16, kWK = kWarps;    // warps along K, and later along N
    static constexpr int kRC = 16 * JT;               // ranks of a pass over K
    static constexpr int kPartPitch = kRC + 8;        // floats; 8 mod 32 spreads 4 rows' pairs over all banks
    static constexpr int kStep = JT <= 2 ? 64 : 32;   // of K at a time
    // Two steps are a turn; after kChain of them (16 products into an accumulator, 32 where there are many) a warp adds its sums
    // to those in shared memory, as the tensor cores cut sums off instead of rounding them (float32 Y, 2000 rows of 100
    // adapters, K = 8192: off by 3.8e-7 in f16 and 2.7e-7 in bf16 at rank 16, a float32 product by 4.5e-7 and 2.1e-7; without
    // it by 1.3e-6 and 1.1e-6). So are the second product's at ranks above 128, two items at a time. What it costs: nothing at ranks up to 32, 2 % at
    // 64 and 128 (6000 x 8192 x 8192 of 200 adapters 342 -> 347 us), 7 % above (4099 x 2560 x 2560, bf16 to float32, 111 -> 118).
    static constexpr int kChain = (JT <= 2 ? 16 : 32) / (2 * kStep / 16);
    __host__ __device__ static int ranks(int R) { return (R + 15) / 16 * 16; }
    static size_t smem(int R, int terms) {
        return shared_floats(R) * 4 + (size_t)kRows * (ranks(R) + 8) * 4 + (size_t)(ranks(R) / 16) * terms * 512 + kRows * 4;
    }
    // the warps' parts of H, and later, when those have been added up, H of all of K
    __host__ __device__ static int shared_floats(int R) {
        const int part = kWK * kRows * kPartPitch, all = kRows * (ranks(R) + 8);
        return part > all ? part : all;
    }
};

template <bool BF, int YDT, int JT, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) lora_kernel(const Params p) {
    using S = Shape<JT>;
    constexpr int kNT = 2 * JT, kXV = S::kStep / 32, kTerms = terms_of(BF, YDT);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ TileSearch s_tile;
    __shared__ int s_row[kThreads], s_rank[kThreads];
    __shared__ float s_scale[kThreads];
    const LoraArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int wk = warp;
    // (blocks is a power of two, of 8 at most: shifts, as a 64-bit division takes 330 cycles)
    const int blocks = (int)cluster_size(), shift = __ffs(blocks) - 1, rank_in = blocks > 1 ? (int)cluster_rank() : 0;
    const int pitch = S::ranks(a.R) + 8;
    float* part = reinterpret_cast<float*>(smem);                           // [kWK][kRows][kPartPitch]
    float* sum = part;                                                      // [kRows][pitch], all of K
    float* h = part + S::shared_floats(a.R);                                // [kRows][pitch], this block's part of K
    uint4* frag = reinterpret_cast<uint4*>(h + S::kRows * pitch);           // [ranks / 16][terms][32]
    uint32_t* top = reinterpret_cast<uint32_t*>(frag + (S::ranks(a.R) / 16) * kTerms * 32);   // [kRows]
    grid_wait();
    grid_release();
    // A batch of a row a thread at most has its rows' numbers on the way while it looks for the tile.
    // So have the ranks and scales of as many adapters.
    const bool few = a.M <= kThreads && a.L <= kThreads;
    if (few) {
        s_row[tid] = tid < a.M ? load(a.row + tid) : -1;
        s_rank[tid] = a.rank && tid < a.L ? load(a.rank + tid) : a.R;
        s_scale[tid] = a.scale && tid < a.L ? load(a.scale + tid) : 1.f;
    }
    int l, from, count;
    if (!find_tile(a, blockIdx.x >> shift, S::kRows, s_tile, l, from, count)) return;      // the whole cluster
    // this lane's two rows
    int m[2], rank;
    float scale;
    if (few) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = g + 8 * i < count ? s_row[from + g + 8 * i] : -1;
        scale = s_scale[l];
        rank = s_rank[l];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = g + 8 * i < count ? load(a.row + from + g + 8 * i) : -1;
        scale = a.scale ? load(a.scale + l) : 1.f;
        rank = a.rank ? load(a.rank + l) : a.R;
    }
    rank = min(max(rank, 0), a.R);
    if (rank == 0) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (m[i] >= a.M) m[i] = -1;

    // ---- H = X A^T, kRC ranks a pass; the block's part of K, its warps' parts of that
    {
        const uint16_t* X = static_cast<const uint16_t*>(a.X);
        const uint16_t* x0 = X + (long long)max(m[0], 0) * a.ldx;
        const uint16_t* x1 = X + (long long)max(m[1], 0) * a.ldx;
        const int steps = a.K / S::kStep;
        const int s0 = steps * rank_in >> shift, s1 = steps * (rank_in + 1) >> shift;     // (K <= 2^30)
        // Two steps are in flight, each in registers of its own: with one set, copied before the next step's loads, each
        // step waited for its own (64 rows of 64 adapters 11.8 -> 10 us).
        uint4 x[2][2][kXV], w[2][kNT][kXV];
        auto fetch = [&](int r0, int s, uint4 (&x)[2][kXV], uint4 (&w)[kNT][kXV]) {
            if (r0 >= rank || s >= s1) return;
            const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((size_t)l * a.R + r0 + g) * a.K;
#pragma unroll
            for (int v = 0; v < kXV; ++v) {
                const size_t k = (size_t)s * S::kStep + v * 32 + q * 8;
#pragma unroll
                for (int n = 0; n < kNT; ++n)
                    load_if(w[n][v], A + (size_t)n * 8 * a.K + k, r0 + n * 8 + g < rank);
                load_if(x[0][v], x0 + k, m[0] >= 0);
                load_if(x[1][v], x1 + k, m[1] >= 0);
            }
        };
        fetch(0, s0 + wk, x[0], w[0]);
        fetch(0, s0 + wk + S::kWK, x[1], w[1]);
        for (int r0 = 0; r0 < rank; r0 += S::kRC) {
            float acc[kNT][4];
            float* const mine = part + (wk * S::kRows + g) * S::kPartPitch + 2 * q;
            auto clear = [&]() {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            };
            // to this lane's place in the warp's part of H, or what is there already
            auto put = [&](bool add) {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float2* to = reinterpret_cast<float2*>(mine + i * 8 * S::kPartPitch + n * 8);
                        const float2 v = add ? *to : make_float2(0.f, 0.f);
                        *to = make_float2(v.x + acc[n][2 * i], v.y + acc[n][2 * i + 1]);
                    }
            };
            clear();
            if (r0 > 0) __syncthreads();        // the pass before has been read
            auto step = [&](const uint4 (&x)[2][kXV], const uint4 (&w)[kNT][kXV]) {
#pragma unroll
                for (int v = 0; v < kXV; ++v)
#pragma unroll
                    for (int n = 0; n < kNT; ++n) {
                        mma<BF>(acc[n], make_uint4(x[0][v].x, x[1][v].x, x[0][v].y, x[1][v].y), w[n][v].x, w[n][v].y);
                        mma<BF>(acc[n], make_uint4(x[0][v].z, x[1][v].z, x[0][v].w, x[1][v].w), w[n][v].z, w[n][v].w);
                    }
            };
            int s = s0 + wk;
            auto turns = [&]() { return (s - s0 - wk) / (2 * S::kWK); };
            for (; s < s1; s += 2 * S::kWK) {
                step(x[0], w[0]);
                fetch(r0, s + 2 * S::kWK, x[0], w[0]);
                if (s + S::kWK >= s1) break;
                step(x[1], w[1]);
                fetch(r0, s + 3 * S::kWK, x[1], w[1]);
                if (turns() % S::kChain == S::kChain - 1) {
                    put(turns() >= S::kChain);
                    clear();
                }
            }
            fetch(r0 + S::kRC, s0 + wk, x[0], w[0]);
            fetch(r0 + S::kRC, s0 + wk + S::kWK, x[1], w[1]);
            put(turns() >= S::kChain);
            __syncthreads();
            constexpr int kWidth = S::kRC / 4;
            for (int i = tid; i < S::kRows * kWidth; i += kThreads) {
                const int row = i / kWidth, c = i % kWidth * 4;
                if (r0 + c >= pitch - 8) continue;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < S::kWK; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(part + (k * S::kRows + row) * S::kPartPitch + c);
                    v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                }
                *reinterpret_cast<float4*>(h + row * pitch + r0 + c) = v;
            }
        }
    }
    if (tid < S::kRows) top[tid] = 0u;

    // ---- the second product's first operands come while the blocks meet
    const int units = (a.N + 31) / 32;
    const int u0 = units * rank_in >> shift, u1 = units * (rank_in + 1) >> shift;         // (N <= 2^30)
    const int chunks = (rank + 15) / 16;
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (size_t)l * a.N * a.R;
    // Items of JT chunks of a unit of 32 columns, two in flight in registers of their own (Y's rows of the second where
    // registers allow it).
    constexpr int kYSets = JT == 4 && YDT == DT_F32 ? 1 : 2;
    uint2 b[2][JT][4];
    Eight<YDT> y[kYSets][2];
    // ranks 16 (c0 + j) + 4 q .. + 3 of the columns of unit u
    auto fetch_b = [&](int u, int c0, uint2 (&b)[JT][4]) {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            const int r = (c0 + j) * 16 + q * 4;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int n = u * 32 + (WIDE ? (g >> 1) * 8 + t * 2 + (g & 1) : t * 8 + g);
                load_if(b[j][t], B + (size_t)n * a.R + r, r < rank && n < a.N);
            }
        }
    };
    auto y_row = [&](int i) { return static_cast<uint8_t*>(a.Y) + (long long)m[i] * a.ldy * (YDT == DT_F32 ? 4 : 2); };
    auto fetch_y = [&](int u, Eight<YDT> (&y)[2]) {
        if constexpr (!WIDE) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (m[i] >= 0) fetch_pairs<YDT>(y[i], y_row(i), u * 32 + q * 2, a.N);
            return;
        }
        if (u * 32 + q * 8 + 8 > a.N) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (m[i] >= 0) y[i].fetch(a.Y, (size_t)((long long)m[i] * a.ldy) + u * 32 + q * 8);
    };
    int next_u = u0 + wk, next_c = 0;       // the item to fetch
    auto fetch_item = [&](uint2 (&b)[JT][4], Eight<YDT> (&y)[2]) {
        if (next_u >= u1) return;
        fetch_b(next_u, next_c, b);
        next_c += JT;
        if (next_c >= chunks) {             // the unit's last
            if (kYSets == 2) fetch_y(next_u, y);
            next_c = 0;
            next_u += S::kWK;
        }
    };
    if (kYSets == 1 && u0 + wk < u1) fetch_y(u0 + wk, y[0]);
    fetch_item(b[0], y[0]);
    fetch_item(b[1], y[kYSets - 1]);

    // ---- H of all of K, in the same order in every block, and its terms
    if (blocks > 1) cluster_sync();
    else __syncthreads();
    join_h<BF, S::kRC / 4>(h, sum, top, pitch, S::kRows, chunks, blocks);
    if (blocks > 1) cluster_arrive();       // waited for at the end
    __syncthreads();
    make_terms<BF, kTerms>(sum, top, frag, pitch, rank, chunks);
    __syncthreads();

    // ---- Y += scale H B^T
    float mul[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) mul[i] = BF ? 1.f : row_unit(top[g + 8 * i]);
    // Two items' products (each item's small terms first) are added up by themselves, and then to the unit's, which wait in H's
    // place (see kChain).
    float acc[4][4];
    float4* const total = reinterpret_cast<float4*>(part) + warp * 4 * 32 + lane;
    int u = u0 + wk, c0 = 0;
    auto item = [&](uint2 (&b)[JT][4], Eight<YDT> (&y)[2]) {
        if (c0 % (2 * JT) == 0)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            if (c0 + j >= chunks) break;
#pragma unroll
            for (int k = kTerms - 1; k >= 0; --k) {
                const int left = rank - (c0 + j) * 16 - q * 4;
                if (k == kTerms - 1 && left < 4)        // values past the adapter's rank are cleared
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        b[j][t].x &= left >= 2 ? ~0u : (left == 1 ? 0xFFFFu : 0u);
                        b[j][t].y &= left == 3 ? 0xFFFFu : 0u;
                    }
                const uint4 h = frag[((c0 + j) * kTerms + k) * 32 + lane];
#pragma unroll
                for (int t = 0; t < 4; ++t) mma<BF>(acc[t], h, b[j][t].x, b[j][t].y);
            }
        }
        c0 += JT;
        if (JT == 4 && chunks > 2 * JT && (c0 % (2 * JT) == 0 || c0 >= chunks))
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (c0 > 2 * JT) {
                    const float4 v = total[t * 32];
                    acc[t][0] += v.x; acc[t][1] += v.y; acc[t][2] += v.z; acc[t][3] += v.w;
                }
                if (c0 < chunks) total[t * 32] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
            }
        if (c0 < chunks) return;
        c0 = 0;
        const int n = u * 32 + q * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (m[i] < 0) continue;
            float d[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                d[2 * t] = acc[t][2 * i] * mul[i];
                d[2 * t + 1] = acc[t][2 * i + 1] * mul[i];
            }
            if (!WIDE || n + 8 <= a.N) {
                float v[8];
                y[i].values(v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = fmaf(scale, d[k], v[k]);
                y[i].round_from(v);
                if constexpr (WIDE) y[i].store(y_row(i), n);
                else store_pairs<YDT>(y[i], y_row(i), u * 32 + q * 2, a.N);
            } else {
                add_edge<YDT>(y_row(i) + n * (size_t)(YDT == DT_F32 ? 4 : 2), d, scale, a.N - n);
            }
        }
        u += S::kWK;
        if (kYSets == 1 && u < u1) fetch_y(u, y);
    };
    while (u < u1) {
        item(b[0], y[0]);
        fetch_item(b[0], y[0]);
        if (u >= u1) break;
        item(b[1], y[kYSets - 1]);
        fetch_item(b[1], y[kYSets - 1]);
    }
    if (blocks > 1) cluster_wait();         // no block leaves while its H is read
}

template <bool BF, int YDT, int JT, bool WIDE>
cudaError_t launch(const LoraArgs& a, int blocks, cudaStream_t s) {
    const Params p{a};
    const size_t smem = Shape<JT>::smem(a.R, terms_of(BF, YDT));
    auto kern = lora_kernel<BF, YDT, JT, WIDE>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // at most one tile that is not full for each adapter that has rows
    const long long tiles = (long long)a.M / Shape<JT>::kRows + (a.L < a.M ? a.L : a.M);
    return launch_behind(kern, dim3((unsigned)(tiles * blocks)), dim3(kThreads), smem, (unsigned)blocks, s, p);
}

}  // namespace lora
}  // namespace qg
