// Low-rank adapters beside a shared projection: Y[m] += scale_l B_l (A_l X[m]) for the rows of every adapter, in one
// launch. This file has the kernel for few rows, lora_many.cuh the one for many; instantiated for f16 (lora_f16.cu) and
// bf16 (lora_bf16.cu).
//
// A cluster of thread blocks takes up to 16 rows of one adapter. Its blocks share K in the first product (H = X A^T,
// R values a row), join their parts of H in distributed shared memory, each in the same order, and share N in the
// second one (H B^T), so neither product needs scratch memory or a second launch. What bounds it is a chain of round
// trips: the offsets, the rows' numbers, the first product's operands, the join, the store. 16 rows of 16 adapters,
// 4096 x 4096 at rank 16: 5.9 us in a graph (the same with next to no K and N: 4.3); 77 rows of 24 adapters of ranks up
// to 64, 9728 x 2560, float32 Y: 16 us.
//
// Both products run on 16x8x16 tensor-core steps from registers, without a copy through shared memory: the order of
// the summed index is free as long as both operands keep to it, so a lane takes 16 neighbouring bytes of a row as its
// values of two steps; and the order of the columns of the second product is chosen so that a lane ends with 8
// neighbouring values of Y's row.
//
// H is exact to float32's rounding where it matters: it enters the second product as a sum of 16-bit terms (hi = its
// nearest 16-bit value, then the nearest to what is left), 2 of them for 16-bit Y (17 bits of bf16, 22 of f16) and 3 of
// bf16 for float32 Y. f16 terms are of H scaled by a power of two for each row, so that they neither overflow nor
// lose their second term to f16's smallest exponent.
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
// 16 x 8 = 16 x 16 * 16 x 8
template <bool BF>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
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

// f16 terms are of H over the power of two of the row's largest |H| (its bits): this is that power.
__device__ __forceinline__ float row_unit(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255u ? 1.f : __uint_as_float(min(max(e, 1u), 253u) << 23);
}
__device__ __forceinline__ float row_unit_inverse(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255u ? 1.f : __uint_as_float((254u - min(max(e, 1u), 253u)) << 23);
}

// H of all of K from the blocks' parts h, added in rank order: [rows][pitch], 16 * chunks columns; top: the bits of each
// row's largest |H| (f16; cleared before). Every thread of the block calls it.
template <bool BF>
__device__ __forceinline__ void join_h(const float* h, float* sum, uint32_t* top, int pitch, int rows, int chunks, int blocks) {
    const int width = chunks * 4;
    for (int i = threadIdx.x; i < rows * width; i += kThreads) {
        const int row = i / width, at = row * pitch + i % width * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (blocks > 1) {
            for (int k0 = 0; k0 < blocks; k0 += 4) {
                float4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < blocks) o[k] = ld_cluster_f32x4(in_block(h + at, k0 + k));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < blocks) {
                        v.x += o[k].x; v.y += o[k].y; v.z += o[k].z; v.w += o[k].w;
                    }
            }
        } else {
            v = *reinterpret_cast<const float4*>(h + at);
        }
        *reinterpret_cast<float4*>(sum + at) = v;
        if constexpr (!BF) {
            const float t = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
            atomicMax(top + row, __float_as_uint(t));
        }
    }
}
// H's 16-bit terms, in the order in which the lanes take them: frag [tiles of 16 rows][chunks][terms][32].
template <bool BF, int TERMS>
__device__ __forceinline__ void make_terms(const float* sum, const uint32_t* top, uint4* frag, int pitch, int tiles, int chunks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    for (int f = warp; f < tiles * chunks; f += kWarps) {
        float v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = f / chunks * 16 + g + 8 * i;
            const float4 o = *reinterpret_cast<const float4*>(sum + row * pitch + f % chunks * 16 + q * 4);
            const float by = BF ? 1.f : row_unit_inverse(top[row]);
            v[i][0] = o.x * by; v[i][1] = o.y * by; v[i][2] = o.z * by; v[i][3] = o.w * by;
        }
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
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= n) break;
        const float v = fmaf(scale, d[k], load_as_float<YDT>(y, k));
        if constexpr (YDT == DT_F32) static_cast<float*>(y)[k] = v;
        else if constexpr (YDT == DT_F16) static_cast<__half*>(y)[k] = __float2half_rn(v);
        else static_cast<__nv_bfloat16*>(y)[k] = __float2bfloat16_rn(v);
    }
}

// The q-th tile of `rows` rows over the adapters: its adapter, first position in `row`, and rows. Offsets are held to
// [0, M] and to the largest before them. Every thread of the block calls it.
//
// Up to 32 adapters each warp looks by itself; more are shared between the block's threads, neighbouring adapters a
// thread (128 rows of 1000 adapters 21 us; with 32 at a time in every warp 34).
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

// Sixteen ranks at a time are a chunk; JT of them are in registers together.
template <int JT>
struct Shape {
    static constexpr int kRows = 16, kWK = kWarps;    // warps along K, and later along N
    static constexpr int kRC = 16 * JT;               // ranks of a pass over K
    static constexpr int kPartPitch = kRC + 8;        // floats; 8 mod 32 spreads 4 rows' pairs over all banks
    static constexpr int kStep = JT <= 2 ? 64 : 32;   // of K at a time
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

template <bool BF, int YDT, int JT>
__global__ void __launch_bounds__(kThreads, 2) lora_kernel(const Params p) {
    using S = Shape<JT>;
    constexpr int kNT = 2 * JT, kXV = S::kStep / 32, kTerms = terms_of(BF, YDT);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ TileSearch s_tile;
    const LoraArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int wk = warp;
    const int blocks = (int)cluster_size(), rank_in = blocks > 1 ? (int)cluster_rank() : 0;
    const int pitch = S::ranks(a.R) + 8;
    float* part = reinterpret_cast<float*>(smem);                           // [kWK][kRows][kPartPitch]
    float* sum = part;                                                      // [kRows][pitch], all of K
    float* h = part + S::shared_floats(a.R);                                // [kRows][pitch], this block's part of K
    uint4* frag = reinterpret_cast<uint4*>(h + S::kRows * pitch);           // [ranks / 16][terms][32]
    uint32_t* top = reinterpret_cast<uint32_t*>(frag + (S::ranks(a.R) / 16) * kTerms * 32);   // [kRows]
    grid_wait();
    grid_release();
    int l, from, count;
    if (!find_tile(a, blockIdx.x / blocks, S::kRows, s_tile, l, from, count)) return;      // the whole cluster
    const int rank = a.rank ? min(max(load(a.rank + l), 0), a.R) : a.R;
    if (rank == 0) return;
    const float scale = a.scale ? load(a.scale + l) : 1.f;

    // this lane's two rows
    int m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = g + 8 * i;
        m[i] = at < count ? load(a.row + from + at) : -1;
        if (m[i] >= a.M) m[i] = -1;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);

    // ---- H = X A^T, kRC ranks a pass; the block's part of K, its warps' parts of that
    {
        const uint16_t* X = static_cast<const uint16_t*>(a.X);
        const uint16_t* x0 = X + (long long)max(m[0], 0) * a.ldx;
        const uint16_t* x1 = X + (long long)max(m[1], 0) * a.ldx;
        const int steps = a.K / S::kStep;
        const int s0 = (int)((long long)steps * rank_in / blocks), s1 = (int)((long long)steps * (rank_in + 1) / blocks);
        for (int r0 = 0; r0 < rank; r0 += S::kRC) {
            const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((size_t)l * a.R + r0 + g) * a.K;
            float acc[kNT][4];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            uint4 x[2][kXV], w[kNT][kXV];
            auto fetch = [&](int s) {
#pragma unroll
                for (int v = 0; v < kXV; ++v) {
                    const size_t k = (size_t)s * S::kStep + v * 32 + q * 8;
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
                        w[n][v] = r0 + n * 8 + g < rank ? load(reinterpret_cast<const uint4*>(A + (size_t)n * 8 * a.K + k)) : zero;
                    x[0][v] = m[0] >= 0 ? load(reinterpret_cast<const uint4*>(x0 + k)) : zero;
                    x[1][v] = m[1] >= 0 ? load(reinterpret_cast<const uint4*>(x1 + k)) : zero;
                }
            };
            if (s0 + wk < s1) fetch(s0 + wk);
            for (int s = s0 + wk; s < s1; s += S::kWK) {
                uint4 cx[2][kXV], cw[kNT][kXV];
#pragma unroll
                for (int v = 0; v < kXV; ++v) {
                    cx[0][v] = x[0][v];
                    cx[1][v] = x[1][v];
#pragma unroll
                    for (int n = 0; n < kNT; ++n) cw[n][v] = w[n][v];
                }
                if (s + S::kWK < s1) fetch(s + S::kWK);
#pragma unroll
                for (int v = 0; v < kXV; ++v)
#pragma unroll
                    for (int n = 0; n < kNT; ++n) {
                        mma<BF>(acc[n], make_uint4(cx[0][v].x, cx[1][v].x, cx[0][v].y, cx[1][v].y), cw[n][v].x, cw[n][v].y);
                        mma<BF>(acc[n], make_uint4(cx[0][v].z, cx[1][v].z, cx[0][v].w, cx[1][v].w), cw[n][v].z, cw[n][v].w);
                    }
            }
            if (r0 > 0) __syncthreads();        // the pass before has been read
            float* mine = part + (wk * S::kRows + g) * S::kPartPitch + 2 * q;
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                *reinterpret_cast<float2*>(mine + n * 8) = make_float2(acc[n][0], acc[n][1]);
                *reinterpret_cast<float2*>(mine + 8 * S::kPartPitch + n * 8) = make_float2(acc[n][2], acc[n][3]);
            }
            __syncthreads();
            const int width = min(S::kRC, pitch - 8 - r0) / 4;
            for (int i = tid; i < S::kRows * width; i += kThreads) {
                const int row = i / width, c = i % width * 4;
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
    const int u0 = (int)((long long)units * rank_in / blocks), u1 = (int)((long long)units * (rank_in + 1) / blocks);
    const int chunks = (rank + 15) / 16;
    const uint16_t* B = static_cast<const uint16_t*>(a.B) + (size_t)l * a.N * a.R;
    const bool wide = a.ldy % (YDT == DT_F32 ? 4 : 8) == 0;
    uint2 b[JT][4];
    Eight<YDT> y[2];
    // ranks 16 (c0 + j) + 4 q .. + 3 of the columns of unit u: bits past the adapter's rank are cleared
    auto fetch_b = [&](int u, int c0) {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            const int r = (c0 + j) * 16 + q * 4, left = rank - r;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int n = u * 32 + (g >> 1) * 8 + t * 2 + (g & 1);
                b[j][t] = left > 0 && n < a.N ? load(reinterpret_cast<const uint2*>(B + (size_t)n * a.R + r)) : make_uint2(0, 0);
                if (left < 4) {
                    b[j][t].x &= left >= 2 ? ~0u : (left == 1 ? 0xFFFFu : 0u);
                    b[j][t].y &= left == 3 ? 0xFFFFu : 0u;
                }
            }
        }
    };
    auto fetch_y = [&](int u) {
        if (!wide || u * 32 + q * 8 + 8 > a.N) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (m[i] >= 0) y[i].fetch(a.Y, (size_t)((long long)m[i] * a.ldy) + u * 32 + q * 8);
    };
    if (u0 + wk < u1) {
        fetch_b(u0 + wk, 0);
        fetch_y(u0 + wk);
    }

    // ---- H of all of K, in the same order in every block, and its terms
    if (blocks > 1) cluster_sync();
    else __syncthreads();
    join_h<BF>(h, sum, top, pitch, S::kRows, chunks, blocks);
    if (blocks > 1) cluster_arrive();       // waited for at the end
    __syncthreads();
    make_terms<BF, kTerms>(sum, top, frag, pitch, 1, chunks);
    __syncthreads();

    // ---- Y += scale H B^T
    float mul[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) mul[i] = BF ? 1.f : row_unit(top[g + 8 * i]);
    for (int u = u0 + wk; u < u1; u += S::kWK) {
        float acc[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
        Eight<YDT> cy[2] = {y[0], y[1]};
        for (int c0 = 0; c0 < chunks; c0 += JT) {
            uint2 cb[JT][4];
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t) cb[j][t] = b[j][t];
            if (c0 + JT < chunks) {
                fetch_b(u, c0 + JT);
            } else if (u + S::kWK < u1) {
                fetch_b(u + S::kWK, 0);
                fetch_y(u + S::kWK);
            }
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                if (c0 + j >= chunks) break;
                const uint4* f = frag + (c0 + j) * kTerms * 32 + lane;
#pragma unroll
                for (int k = 0; k < kTerms; ++k) {
                    const uint4 w = f[k * 32];
#pragma unroll
                    for (int t = 0; t < 4; ++t) mma<BF>(acc[t], w, cb[j][t].x, cb[j][t].y);
                }
            }
        }
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
            uint8_t* out = static_cast<uint8_t*>(a.Y) + ((long long)m[i] * a.ldy + n) * (YDT == DT_F32 ? 4 : 2);
            if (wide && n + 8 <= a.N) {
                float v[8];
                cy[i].values(v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = fmaf(scale, d[k], v[k]);
                cy[i].round_from(v);
                cy[i].store(out, 0);
            } else {
                add_edge<YDT>(out, d, scale, a.N - n);
            }
        }
    }
    if (blocks > 1) cluster_wait();         // no block leaves while its H is read
}

template <bool BF, int YDT, int JT>
cudaError_t launch(const LoraArgs& a, int blocks, cudaStream_t s) {
    const Params p{a};
    const size_t smem = Shape<JT>::smem(a.R, terms_of(BF, YDT));
    auto kern = lora_kernel<BF, YDT, JT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // at most one tile that is not full for each adapter that has rows
    const long long tiles = (long long)a.M / Shape<JT>::kRows + (a.L < a.M ? a.L : a.M);
    return launch_behind(kern, dim3((unsigned)(tiles * blocks)), dim3(kThreads), smem, (unsigned)blocks, s, p);
}

}  // namespace lora
}  // namespace qg
