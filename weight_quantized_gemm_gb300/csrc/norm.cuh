// The step between two blocks of a model, in one pass over the rows: the norm behind a block, its gate, the residual
// sum, and the norm in front of the next block. Formulas and conventions: include/qgemm.h. Instantiated for each type
// of X (norm_f32.cu, norm_f16.cu, norm_bf16.cu).
//
// Every input and output byte moves once, so HBM bounds long batches and the launch short ones. A row's values stay
// in registers, in float32, from the first load to the last store: a thread holds CH pieces of 8 neighbouring values,
// and both norms are reductions over the row's threads. The mean square of centred values (LAYER) takes a second
// reduction and not the difference of two sums, which loses the digits that a large mean shares.
//
// A thread holds as much as keeps enough blocks on an SM that loads are in flight while others wait for their sums:
// CH = 4 with 128 threads and 6 blocks an SM at K = 4096 (16384 rows in bf16 with both norms, gate and residual:
// 83 us, 6.5 TB/s). The same with 2 pieces a thread and 4 blocks of 256: 92 us (more instructions a value: sums,
// barriers and addresses are a thread's, not a value's), with 16 pieces and a warp a row 161 us (4 warps on an SM),
// rows prefetched through shared memory 100 us and more (the weights then miss L1). A few rows are spread over more
// threads, where the chain of the two sums is the time (4 rows: 1.8 us).
#pragma once

#include "serve.cuh"

namespace qg {
namespace norm {

// Threads of a block at most, and blocks an SM at least (which bounds the registers): of rows above 5120 and up to 8192
// values three blocks or more (16384 x 8192 in bf16, 80 registers a thread, 195 -> 170 us; x 6144 138 -> 126). Three blocks of the next longer
// rows lose more to the stack than they gain (x 9728 222 us with two blocks, 241 with three); above 10240 values the bound of 1024 threads leaves
// 64 registers, and 200 to 360 bytes a thread on the stack (instances for 384 or 512 threads were not tried). But with a residual in float32 that
// is asked for only where it is added (kLate): 1023 x 9728 36.4 -> 34.4 us, x 8192 32.9 -> 26.6, x 6144 25.8 -> 21.1,
// 2000 x 16384 119 -> 92; rows up to 5120 lose by that (20.8 -> 22.2).
template <int SDT, int MAXT>
constexpr int kBlocks = MAXT <= 128 ? 6 : (MAXT <= 192 ? 4 : (MAXT <= 256 ? 3 : (MAXT <= 320 ? (SDT == DT_F32 ? 3 : 2) : 1)));

template <int XDT, int SDT, int YDT, int CH, int MAXT>
__global__ void __launch_bounds__(MAXT, kBlocks<SDT, MAXT>) norm_kernel(const NormArgs a, const float per) {
    // a slot for each reduction, so that one barrier each is enough
    __shared__ __align__(16) float part[4][32];
    const int t = threadIdx.x, threads = blockDim.x, warps = threads >> 5, pieces = a.K >> 3;
    const long long m = blockIdx.x;
    if (warps > 1) {
        if (t < 32)
#pragma unroll
            for (int q = 0; q < 4; ++q) part[q][t] = 0.f;
        __syncthreads();
    }
    grid_wait();
    grid_release();
    float f[CH][8];
    Eight<XDT> x[CH], gate[CH];
    constexpr bool kLate = SDT == DT_F32 && MAXT > 192 && CH > 1;
    Eight<SDT> res[kLate ? 1 : CH];
    bool live[CH];
    {
        const size_t x0 = (size_t)(m * a.ldx), r0 = (size_t)(m * a.K), g0 = (size_t)(m * a.ldg);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int p = c * threads + t;
            live[c] = c < CH - 1 || p < pieces;      // (the launch has (CH - 1) * threads <= pieces)
            if (live[c]) x[c].fetch(a.X, x0 + p * 8);
            else x[c] = Eight<XDT>{};           // adds nothing to the sums
        }
        if (!kLate && a.residual)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (live[c]) res[kLate ? 0 : c].fetch(a.residual, r0 + (c * threads + t) * 8);
        if (a.gate)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (live[c]) gate[c].fetch(a.gate, g0 + (c * threads + t) * 8);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) x[c].values(f[c]);
    auto total = [&](float v, int slot) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) return v;
        if ((t & 31) == 0) part[slot][t >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int q = 0; q < warps; q += 4) {        // (slots past the last warp's hold 0)
            const float4 p = *reinterpret_cast<const float4*>(&part[slot][q]);
            v += (p.x + p.y) + (p.z + p.w);
        }
        return v;
    };
    // The factor of the norm of the row; LAYER leaves its centred values in f.
    auto norm = [&](int slot) {
        if (a.kind == NORM_LAYER) {
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += f[c][j];
            // sum / K: the product with the rounded 1 / K, refined once by its residual. Without that it is off where the
            // quotient is exact, and a row of 12345 is not 0 but -0.3 at K = 3584 and eps = 1e-5.
            const float all = total(sum, slot), about = all * per;
            const float mean = fmaf(fmaf(-about, (float)a.K, all), per, about);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[c][j] = live[c] ? f[c][j] - mean : 0.f;
        }
        float sum = 0.f, other = 0.f;       // two chains
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                sum = fmaf(f[c][j], f[c][j], sum);
                other = fmaf(f[c][j + 1], f[c][j + 1], other);
            }
        return rsqrtf(fmaf(total(sum + other, slot + 1), per, a.eps));
    };
    const float by = a.post ? norm(0) * a.x_scale : a.x_scale;
    const size_t row = (size_t)(m * a.K);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
        const int p = c * threads + t;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[c][j] *= by;
        if (a.post_weight) {
            Eight<DT_F32> w;
            w.fetch(a.post_weight, (size_t)p * 8);
            w.values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] *= v[j];
        }
        if (a.gate) {
            gate[c].values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] *= v[j];
        }
        if (a.residual) {
            if (kLate) res[0].fetch(a.residual, row + p * 8);
            res[kLate ? 0 : c].values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] = fmaf(a.r_scale, v[j], f[c][j]);
        }
        if (a.S) {
            Eight<SDT> out;
            out.round_from(f[c]);
            out.store(a.S, row + p * 8);
        }
    }
    if (!a.Y) return;
    const float inv = norm(2);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
        const int p = c * threads + t;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[c][j] *= inv;
        if (a.weight) {
            Eight<DT_F32> w;
            w.fetch(a.weight, (size_t)p * 8);
            w.values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] *= v[j];
        }
        if (a.bias) {
            Eight<DT_F32> w;
            w.fetch(a.bias, (size_t)p * 8);
            w.values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] += v[j];
        }
        Eight<YDT> out;
        out.round_from(f[c]);
        out.store(a.Y, row + p * 8);
    }
}

inline int threads_of(int pieces, int ch) { return ((pieces + ch - 1) / ch + 31) / 32 * 32; }

template <int XDT, int SDT, int YDT, int CH, int MAXT>
cudaError_t launch_ch(const NormArgs& a, cudaStream_t s) {
    return launch_behind(norm_kernel<XDT, SDT, YDT, CH, MAXT>, dim3((unsigned)a.M), dim3(threads_of(a.K / 8, CH)), 0, 1, s, a,
                         1.f / (float)a.K);
}
template <int XDT, int SDT, int YDT>
cudaError_t launch_y(const NormArgs& a, cudaStream_t s) {
    const int pieces = a.K / 8;
    // One piece a thread in rows too short for more, or where an SM takes its share of the rows at once (K = 4096: 304 rows
    // 4.7 us, 400 rows 5.1; with four pieces 400 rows take 7.6).
    const int one = threads_of(pieces, 1), at_once = one < 1536 ? 1536 / one : 0;
    if (pieces < 32 || (pieces <= 1024 && a.M <= kTargetSms * at_once)) return launch_ch<XDT, SDT, YDT, 1, 1024>(a, s);
    // Only a thread's last piece may lie past the row's end: from 32 pieces on with 2 a thread, and with 4 but where a
    // row is little longer than a whole number of its warps' pieces.
    if (3 * threads_of(pieces, 4) > pieces) return launch_ch<XDT, SDT, YDT, 2, 192>(a, s);
    if (pieces <= 4 * 128) return launch_ch<XDT, SDT, YDT, 4, 128>(a, s);
    if (pieces <= 4 * 160) return launch_ch<XDT, SDT, YDT, 4, 160>(a, s);
    if (pieces <= 4 * (SDT == DT_F32 ? 192 : 256)) return launch_ch<XDT, SDT, YDT, 4, 256>(a, s);
    if (pieces <= 4 * 320) return launch_ch<XDT, SDT, YDT, 4, 320>(a, s);
    return launch_ch<XDT, SDT, YDT, 4, 1024>(a, s);
}
template <int XDT, int SDT>
cudaError_t launch_s(const NormArgs& a, int y_dtype, cudaStream_t s) {
    switch (y_dtype) {
        case DT_F32: return launch_y<XDT, SDT, DT_F32>(a, s);
        case DT_F16: return launch_y<XDT, SDT, DT_F16>(a, s);
        default: return launch_y<XDT, SDT, DT_BF16>(a, s);
    }
}
template <int XDT>
cudaError_t launch_x(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s) {
    switch (s_dtype) {
        case DT_F32: return launch_s<XDT, DT_F32>(a, y_dtype, s);
        case DT_F16: return launch_s<XDT, DT_F16>(a, y_dtype, s);
        default: return launch_s<XDT, DT_BF16>(a, y_dtype, s);
    }
}

}  // namespace norm
}  // namespace qg
