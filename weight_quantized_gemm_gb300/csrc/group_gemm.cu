// Products of microscaled 4-bit or 16-bit operands, one (dense) or one per expert over ragged row
// groups: C[m][n] = epilogue(a_scale[m] * b_scale[n] * sum_k A[m][k] B[e(m)][n][k]).
#include "epilogue.cuh"
#include "fp4.cuh"

namespace qg {
namespace {

using namespace fp4;

constexpr int kTile = 64, kChunk = 16;

template <int GF>
__device__ __forceinline__ void load16(const GroupGemmArgs& a, const void* p, const void* scales, bool tiled, size_t row, int local,
                                       int k0, float* x) {
    if constexpr (GF == GF_MXFP4 || GF == GF_NVFP4) {
        const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + (row * a.K + k0) / 2);
        constexpr int B = Format<GF>::kBlock;
        const uint8_t* s = static_cast<const uint8_t*>(scales);
        const uint32_t byte = tiled ? s[tiled_index(local, k0 / B, scale_ktiles(a.K, B))] : s[row * scale_pitch(a.K, B) + k0 / B];
        const float f = GF == GF_MXFP4 ? mx_scale_value(byte) : nv_scale_value(byte);
        unpack8(c.x, x);
        unpack8(c.y, x + 8);
        for (int i = 0; i < 16; ++i) x[i] *= f;
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + row * a.K + k0;
        for (int i = 0; i < 16; ++i)
            x[i] = GF == GF_F16 ? __half2float(__ushort_as_half(q[i])) : __uint_as_float((uint32_t)q[i] << 16);
    }
}

template <int GF>
__global__ void __launch_bounds__(256) group_gemm_kernel(const GroupGemmArgs a) {
    __shared__ float s_a[kTile][kChunk + 1], s_b[kTile][kChunk + 1], s_c[kTile][kTile + 1];
    int e = 0, lo = 0, hi = a.M, mt = blockIdx.y;
    if (a.offsets) {
        for (; e < a.E; ++e) {
            lo = min(max(a.offsets[e], 0), a.M);
            hi = min(max(a.offsets[e + 1], lo), a.M);
            const int tiles = (hi - lo + kTile - 1) / kTile;
            if (mt < tiles) break;
            mt -= tiles;
        }
        if (e == a.E) return;
    }
    const int m0 = lo + mt * kTile, n0 = blockIdx.x * kTile;
    const uint8_t* Bs = a.Bs ? static_cast<const uint8_t*>(a.Bs) + (size_t)e * ((size_t)((a.N + 127) / 128) * scale_ktiles(a.K, GF == GF_MXFP4 ? 32 : 16) * 512) : nullptr;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kChunk) {
        if (threadIdx.x < kTile) {
            const int m = min(m0 + (int)threadIdx.x, hi - 1);
            load16<GF>(a, a.A, a.As, false, m, 0, k0, s_a[threadIdx.x]);
        } else if (threadIdx.x < 2 * kTile) {
            const int r = threadIdx.x - kTile, n = min(n0 + r, a.N - 1);
            load16<GF>(a, a.B, Bs, true, (size_t)e * a.N + n, n, k0, s_b[r]);
        }
        __syncthreads();
        for (int k = 0; k < kChunk; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s_a[threadIdx.x / 16 * 4 + i][k], s_b[threadIdx.x % 16 * 4 + j][k], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + threadIdx.x / 16 * 4 + i, n = n0 + threadIdx.x % 16 * 4 + j;
            float v = acc[i][j];
            if (m < hi && n < a.N) {
                if (a.a_scale) v *= a.a_scale[m];
                if (a.b_scale) v *= a.b_scale[(size_t)e * a.N + n];
                if (a.bias) v += a.bias[(size_t)e * a.N + n];
            }
            s_c[threadIdx.x / 16 * 4 + i][threadIdx.x % 16 * 4 + j] = v;
        }
    __syncthreads();
    const bool glu = a.act == ACT_SWIGLU;
    const int cols = glu ? a.N / 2 : a.N, width = glu ? kTile / 2 : kTile, c0 = glu ? n0 / 2 : n0;
    for (int i = threadIdx.x; i < kTile * width; i += 256) {
        const int r = i / width, c = i % width, m = m0 + r, n = c0 + c;
        if (m >= hi || n >= cols) continue;
        float v = glu ? act_apply(ACT_SILU, s_c[r][2 * c]) * s_c[r][2 * c + 1] : act_apply(a.act, s_c[r][c]);
        const size_t at = (size_t)m * cols + n;
        if (a.residual)
            v += a.c_dtype == DT_F32 ? load_c<DT_F32>(a.residual, at)
                                     : (a.c_dtype == DT_F16 ? load_c<DT_F16>(a.residual, at) : load_c<DT_BF16>(a.residual, at));
        store_out_rt(a.C, at, v, a.c_dtype);
    }
}

}  // namespace

cudaError_t launch_group_gemm(const GroupGemmArgs& a, int fmt, cudaStream_t s) {
    const dim3 grid((a.N + kTile - 1) / kTile, (a.M + kTile - 1) / kTile + (a.offsets ? a.E : 0));
    switch (fmt) {
        case GF_F16: group_gemm_kernel<GF_F16><<<grid, 256, 0, s>>>(a); break;
        case GF_BF16: group_gemm_kernel<GF_BF16><<<grid, 256, 0, s>>>(a); break;
        case GF_MXFP4: group_gemm_kernel<GF_MXFP4><<<grid, 256, 0, s>>>(a); break;
        default: group_gemm_kernel<GF_NVFP4><<<grid, 256, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace qg
