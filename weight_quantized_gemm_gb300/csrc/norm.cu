// The step between two blocks of a model, in one pass over the rows: the norm behind a block, its gate, the residual
// sum, and the norm in front of the next block. Formulas and conventions: include/qgemm.h.
//
// Every input and output byte moves once, so HBM bounds long batches and the launch short ones. A row's values stay
// in registers, in float32, from the first load to the last store: a thread holds CH pieces of 8 neighbouring values,
// and both norms are reductions over the row's threads. The mean square of centred values (LAYER) takes a second
// reduction and not the difference of two sums, which loses the digits that a large mean shares.
#include "serve.cuh"

namespace qg {
namespace {

template <int XDT, int SDT, int YDT, int CH>
__global__ void __launch_bounds__(CH == 4 ? 1024 : 512) norm_kernel(const NormArgs a) {
    __shared__ float part[4][32];       // a slot for each reduction, so that one barrier each is enough
    const int t = threadIdx.x, threads = blockDim.x, warps = threads >> 5, pieces = a.K >> 3;
    const bool in = (long long)blockIdx.x * blockDim.y + threadIdx.y < a.M;
    const size_t m = in ? (size_t)blockIdx.x * blockDim.y + threadIdx.y : 0;
    grid_wait();
    grid_release();
    // A piece past the row's end stays zero and is not counted.
    Eight<XDT> x[CH], gate[CH];
    Eight<SDT> res[CH];
    bool live[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int p = c * threads + t;
        live[c] = in && p < pieces;
        if (!live[c]) continue;
        x[c].fetch(a.X, m * a.ldx + p * 8);
        if (a.residual) res[c].fetch(a.residual, m * a.K + p * 8);
        if (a.gate) gate[c].fetch(a.gate, m * a.ldg + p * 8);
    }
    auto total = [&](float v, int slot) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) return v;
        float* mine = part[slot] + threadIdx.y * warps;
        if ((t & 31) == 0) mine[t >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < warps; ++w) v += mine[w];
        return v;
    };
    float f[CH][8];
    const float per = 1.f / (float)a.K;
    // (f - mean) * inv is the norm of the row
    auto norm = [&](float& mean, float& inv, int slot) {
        mean = 0.f;
        if (a.kind == NORM_LAYER) {
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (live[c])
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += f[c][j];
            mean = total(sum, slot) * per;
        }
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (live[c])
#pragma unroll
                for (int j = 0; j < 8; ++j) sq = fmaf(f[c][j] - mean, f[c][j] - mean, sq);
        inv = rsqrtf(fmaf(total(sq, slot + 1), per, a.eps));
    };
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (live[c]) x[c].values(f[c]);
    float mean = 0.f, inv = 1.f;
    if (a.post) norm(mean, inv, 0);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
        const int p = c * threads + t;
        if (a.post) {
            Eight<DT_F32> w;
            float v[8];
            if (a.post_weight) {
                w.fetch(a.post_weight, (size_t)p * 8);
                w.values(v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] = (f[c][j] - mean) * inv * (a.post_weight ? v[j] : 1.f);
        }
        if (a.gate) {
            float v[8];
            gate[c].values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] *= v[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[c][j] *= a.x_scale;
        if (a.residual) {
            float v[8];
            res[c].values(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[c][j] = fmaf(a.r_scale, v[j], f[c][j]);
        }
        if (a.S) {
            Eight<SDT> out;
            out.round_from(f[c]);
            out.store(a.S, m * a.K + p * 8);
        }
    }
    if (!a.Y) return;
    norm(mean, inv, 2);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!live[c]) continue;
        const int p = c * threads + t;
        Eight<DT_F32> w, b;
        float v[8], u[8];
        if (a.weight) {
            w.fetch(a.weight, (size_t)p * 8);
            w.values(v);
        }
        if (a.bias) {
            b.fetch(a.bias, (size_t)p * 8);
            b.values(u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[c][j] = fmaf((f[c][j] - mean) * inv, a.weight ? v[j] : 1.f, a.bias ? u[j] : 0.f);
        Eight<YDT> out;
        out.round_from(f[c]);
        out.store(a.Y, m * a.K + p * 8);
    }
}

template <int XDT, int SDT, int YDT>
cudaError_t launch_y(const NormArgs& a, cudaStream_t s) {
    const int pieces = a.K / 8;
    const int ch = pieces <= 512 ? 1 : (pieces <= 1024 ? 2 : 4);
    const int threads = ((pieces + ch - 1) / ch + 31) / 32 * 32;
    const int rows = threads >= 128 ? 1 : 128 / threads;
    const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(threads, rows);
    switch (ch) {
        case 1: return launch_behind(norm_kernel<XDT, SDT, YDT, 1>, grid, block, 0, 1, s, a);
        case 2: return launch_behind(norm_kernel<XDT, SDT, YDT, 2>, grid, block, 0, 1, s, a);
        default: return launch_behind(norm_kernel<XDT, SDT, YDT, 4>, grid, block, 0, 1, s, a);
    }
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

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int x_dtype, int s_dtype, int y_dtype, cudaStream_t s) {
    switch (x_dtype) {
        case DT_F32: return launch_x<DT_F32>(a, s_dtype, y_dtype, s);
        case DT_F16: return launch_x<DT_F16>(a, s_dtype, y_dtype, s);
        default: return launch_x<DT_BF16>(a, s_dtype, y_dtype, s);
    }
}

}  // namespace qg
