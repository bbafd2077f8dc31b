// Microscaled 4-bit quantization (activation rows and [K][N] weights) and its inverse.
//
// Formulas and formats: fp4.cuh and include/qgemm.h. All three kernels move each input and output
// byte once, so HBM bounds them; a thread takes 16 consecutive values of a row (one NVFP4 block, half
// an MXFP4 block, whose two halves are neighbouring lanes), which makes 8 bytes of codes.
// 16384 x 14336 in bf16: MXFP4 91 us (6.5 TB/s), NVFP4 115 us (5.2 TB/s: a row's codes wait for its
// largest value, so loads and stores of a block alternate; four blocks an SM leave it 16 to 20 bytes of
// spills a thread), back 92 us from NVFP4 (6.5 TB/s) and 96 from MXFP4 (6.2); 4 rows 1.5 us in MXFP4 and 3
// in NVFP4, which is the launch and one row's two steps.
#include "experts.cuh"
#include "fp4.cuh"

namespace qg {
namespace {

using namespace fp4;

constexpr int kUnit = 16;   // values per thread

// The 16 values of unit u of a row, as stored.
template <int DT>
struct Raw {
    static constexpr int kVecs = DT == DT_F32 ? 4 : 2;
    uint4 v[kVecs];
    __device__ __forceinline__ void load(const void* row, int u) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)u * kUnit * (DT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = qg::load(p + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    // values 8 h .. 8 h + 7
    __device__ __forceinline__ void eight(int h, float (&x)[8]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v) + h * (DT == DT_F32 ? 8 : 4);
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == DT_F16) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + i));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                } else {
                    x[2 * i] = __uint_as_float(w[i] << 16);
                    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
        }
    }
    // Bits of the largest |x| as float32 (an infinity or NaN is larger than any number): the bits of
    // positive values order as whole numbers do, two 16-bit ones at a time.
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        if constexpr (DT == DT_F32) {
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < kUnit; ++i) t = max(t, w[i] & 0x7FFFFFFFu);
            return t;
        } else {
            constexpr uint32_t kAbs = 0x7FFF7FFFu;
            uint32_t t = w[0] & kAbs;
#pragma unroll
            for (int i = 1; i < kUnit / 2 - 1; i += 2) t = __vimax3_u16x2(t, w[i] & kAbs, w[i + 1] & kAbs);
            t = __vimax3_u16x2(t, w[kUnit / 2 - 1] & kAbs, 0u);
            t = max(t & 0xFFFFu, t >> 16);
            return DT == DT_BF16 ? t << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)t)));
        }
    }
};

// Codes of one NVFP4 block of values x with row factor mul (a power of two) and block scale s: the
// e2m1 value nearest to x * mul / s. The quotient must land on a tie exactly where the value does.
// float32: the correctly rounded quotient does, from the rounded reciprocal of s by one correction step
// (Markstein 1990; s has 4 significant bits). 16-bit values (at most 11 significant bits) are either
// on a tie or at least 2^-13 away from it (ties are 0.25 and more), so x * (mul / s), wrong by a few
// 2^-23, is rounded to a multiple of 2^-16 by adding and subtracting 192, which puts it back on the
// tie or keeps it off.
// r = 1 / s (0 for s = 0); eight values at a time, which keeps the registers that a thread needs low.
template <int DT>
__device__ __forceinline__ uint32_t nv_codes8(const float (&x)[8], float mul, float s, float r) {
    const float rm = r * mul;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (DT == DT_F32) {
            const float y = x[i] * mul, q0 = y * r;
            q[i] = __fmaf_rn(__fmaf_rn(-q0, s, y), r, q0);
        } else {
            q[i] = __fsub_rn(__fmaf_rn(x[i], rm, 192.f), 192.f);
        }
        q[i] = copysignf(q[i], x[i]);
    }
    return mul != 0.f ? pack8(q) : 0u;
}
__device__ __forceinline__ float inverse(float s) { return s > 0.f ? __fdiv_rn(1.f, s) : 0.f; }

struct QuantArgs {
    int M, K;
    const void* X;
    long long ldx_bytes;
    int x_rows;
    const int32_t* rows;      // source row of each output row, or none
    int layout, pitch, ktiles;
    int rows_out, units_out;  // rows and units that have scale bytes (padding included)
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;
};

__device__ __forceinline__ size_t scale_index(const QuantArgs& a, int m, int j) {
    return a.layout == SC_ROWS ? (size_t)m * a.pitch + j : tiled_index(m, j, a.ktiles);
}
// Row m's values (null: a row of zeros: past the end, or gathered from outside X).
__device__ __forceinline__ const uint8_t* source_row(const QuantArgs& a, int m) {
    if (m >= a.M) return nullptr;
    const int r = a.rows ? load(a.rows + m) : m;
    return r >= 0 && r < a.x_rows ? static_cast<const uint8_t*>(a.X) + (long long)r * a.ldx_bytes : nullptr;
}

// MXFP4: every block is by itself. Block: 32 units (512 values) x 8 rows.
template <int DT>
__global__ void __launch_bounds__(256) mx_quant_kernel(const QuantArgs a) {
    grid_wait();
    grid_release();
    const int u = blockIdx.y * 32 + threadIdx.x, m = blockIdx.x * 8 + threadIdx.y;
    if (m >= a.rows_out) return;               // whole warps: a warp is 32 units of one row
    const bool in = m < a.M && u < a.K / kUnit;
    const uint8_t* row = in ? source_row(a, m) : nullptr;
    Raw<DT> raw;
    if (row) raw.load(row, u);
    else raw.zero();
    uint32_t top = raw.top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    float mul;
    const uint32_t byte = mx_scale(top, &mul);
    if (in) {
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
            raw.eight(h, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= mul;
            c[h] = mul != 0.f ? pack8(x) : 0u;
        }
        reinterpret_cast<uint2*>(a.codes)[(size_t)m * (a.K / kUnit) + u] = make_uint2(c[0], c[1]);
    }
    if ((u & 1) == 0 && u < a.units_out) a.scales[scale_index(a, m, u >> 1)] = in ? (uint8_t)byte : (uint8_t)0;
}

// NVFP4: the row's largest value comes first, so each thread keeps kKeep units of the row in
// registers between the two steps (rows of up to 16384 values, float32 8192; the rest of longer ones
// is read again). A row takes as few warps as that allows, and a thread block of kNvThreads as many
// rows as fit: with one row a block, rows of 4096 had one load a thread in flight (17 us for 4096 rows
// against 11). Four blocks an SM: while one computes, the others load.
constexpr int kNvThreads = 256;
template <int DT>
constexpr int kKeep = DT == DT_F32 ? 2 : 4;
template <int DT>
__global__ void __launch_bounds__(kNvThreads, 4) nv_quant_kernel(const QuantArgs a) {
    __shared__ uint32_t s_top[kNvThreads / 32];
    const int units = a.K / kUnit, step = blockDim.x, t = threadIdx.x;      // threads of a row; this one
    const int m = blockIdx.x * blockDim.y + threadIdx.y;
    grid_wait();
    grid_release();
    const uint8_t* row = source_row(a, m);
    Raw<DT> keep[kKeep<DT>];
    uint32_t top = 0;
    if (row) {
#pragma unroll
        for (int i = 0; i < kKeep<DT>; ++i)
            if (t + i * step < units) keep[i].load(row, t + i * step);
            else keep[i].zero();
#pragma unroll
        for (int i = 0; i < kKeep<DT>; ++i) top = max(top, keep[i].top());
        for (int u = t + kKeep<DT> * step; u < units; u += step) {
            Raw<DT> raw;
            raw.load(row, u);
            top = max(top, raw.top());
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const int warps = step / 32;
    if (warps > 1) {
        if ((t & 31) == 0) s_top[threadIdx.y * warps + (t >> 5)] = top;
        __syncthreads();
        for (int w = 0; w < warps; ++w) top = max(top, s_top[threadIdx.y * warps + w]);
    }
    if (m >= a.rows_out) return;
    float mul;
    const float g = nv_row_scale(top, &mul);
    if (t == 0 && m < a.M) a.row_scale[m] = g;
    auto emit = [&](const Raw<DT>& raw, int u) {
        float s;
        const uint32_t most = mul != 0.f ? __float_as_uint(__uint_as_float(raw.top()) * mul) : 0u;
        a.scales[scale_index(a, m, u)] = (uint8_t)nv_scale(most, &s);
        const float r = inverse(s);
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
            raw.eight(h, x);
            c[h] = nv_codes8<DT>(x, mul, s, r);
        }
        reinterpret_cast<uint2*>(a.codes)[(size_t)m * units + u] = make_uint2(c[0], c[1]);
    };
    if (row) {
#pragma unroll
        for (int i = 0; i < kKeep<DT>; ++i)
            if (t + i * step < units) emit(keep[i], t + i * step);
        for (int u = t + kKeep<DT> * step; u < units; u += step) {
            Raw<DT> raw;
            raw.load(row, u);
            emit(raw, u);
        }
    } else if (m < a.M) {
        for (int u = t; u < units; u += step) {
            a.scales[scale_index(a, m, u)] = 0;
            reinterpret_cast<uint2*>(a.codes)[(size_t)m * units + u] = make_uint2(0, 0);
        }
    }
    for (int u = t + (m < a.M ? units : 0); u < a.units_out; u += step) a.scales[scale_index(a, m, u)] = 0;
}

// The inverse: y = code * block scale * row scale in float32, rounded to y's type. code * block scale is
// exact, so float32 rounds once, and not at all where the row scale is a power of two (as nv_row_scale's).
struct DequantArgs {
    int M, K;
    int layout, pitch, ktiles;
    const uint8_t* codes;
    const uint8_t* scales;
    const float* row_scale;
    void* Y;
};
// A thread writes 32 bytes: 16 values, or 8 of float32 (64 bytes a thread took half as long again).
template <int DT>
constexpr int kOut = DT == DT_F32 ? 8 : 16;
template <int FMT, int DT>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const DequantArgs a) {
    constexpr int kN = kOut<DT>;
    grid_wait();
    grid_release();
    const int units = a.K / kN;
    const int u = blockIdx.y * 32 + threadIdx.x, m = blockIdx.x * 8 + threadIdx.y;
    if (m >= a.M || u >= units) return;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes) + ((size_t)m * units + u) * (kN / 8);
    const int j = u * kN / Format<FMT>::kBlock;
    const uint32_t byte = load(a.scales + (a.layout == SC_ROWS ? (size_t)m * a.pitch + j : tiled_index(m, j, a.ktiles)));
    float s = FMT == GF_MXFP4 ? mx_scale_value(byte) : nv_scale_value(byte), g = 1.f;
    if (a.row_scale) {
        g = load(a.row_scale + m);
        // code * s must not overflow where g brings it back (both changes are exact)
        if (FMT == GF_MXFP4 && fabsf(g) < 1.f) {
            s *= 0.25f;
            g *= 4.f;
        }
    }
    float y[kN];
    if constexpr (kN == 16) {
        const uint2 c = load(reinterpret_cast<const uint2*>(codes));
        unpack8(c.x, y);
        unpack8(c.y, y + 8);
    } else {
        unpack8(load(codes), y);
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < kN; ++i) y[i] = y[i] * s * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (DT == DT_F32) {
            w[i] = __float_as_uint(y[i]);
        } else if constexpr (DT == DT_F16) {
            const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    uint4* out = static_cast<uint4*>(a.Y) + ((size_t)m * units + u) * 2;
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// A float32 weight [K][N] to codes [N][K/2] with TILED scales: 32 channels x 64 of K at a time
// through shared memory (reads along N, writes along K); 128 threads, four units a channel. One
// thread block per 32 channels runs through K; NVFP4 runs through it twice, first for the channels'
// largest |w|. Offline work, so it is kept simple: one pass over K by a block behind
// two barriers per 64 values is a chain of load latencies (4096 x 14336: MXFP4 194 us, NVFP4 367).
struct PackArgs {
    const float* W;
    int K, N, ktiles;
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;
};
template <int FMT>
__global__ void __launch_bounds__(128) fp4_pack_kernel(const PackArgs a) {
    __shared__ float s_w[64][33];
    const int n0 = blockIdx.x * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int n = n0 + (int)(threadIdx.x >> 2), g = threadIdx.x & 3;   // this thread's channel and unit
    const int units = a.K / kUnit;
    auto fill = [&](int k0) {
        __syncthreads();
        for (int k = ty; k < 64; k += 4) s_w[k][tx] = n0 + tx < a.N ? a.W[(size_t)(k0 + k) * a.N + n0 + tx] : 0.f;
        __syncthreads();
    };
    float x[kUnit], mul = 1.f;
    auto take = [&]() {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            x[i] = s_w[g * kUnit + i][threadIdx.x >> 2];
            t = max(t, abs_bits(x[i]));
        }
        return t;
    };
    if constexpr (FMT == GF_NVFP4) {
        uint32_t top = 0;
        for (int k0 = 0; k0 < a.K; k0 += 64) {
            fill(k0);
            top = max(top, take());
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float gs = nv_row_scale(top, &mul);
        if (g == 0 && n < a.N) a.row_scale[n] = gs;
    }
    for (int k0 = 0; k0 < a.K; k0 += 64) {
        fill(k0);
        uint32_t top = take();
        const int u = k0 / kUnit + g;
        uint2 c;
        uint32_t byte;
        int j;
        if constexpr (FMT == GF_MXFP4) {
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            byte = mx_scale(top, &mul);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) x[i] *= mul;
            c = mul != 0.f ? make_uint2(pack8(x), pack8(x + 8)) : make_uint2(0, 0);
            j = u >> 1;
        } else {
            float s;
            byte = nv_scale(mul != 0.f ? __float_as_uint(__uint_as_float(top) * mul) : 0u, &s);
            const float r = inverse(s);
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] = x[i];
                hi[i] = x[8 + i];
            }
            c = make_uint2(nv_codes8<DT_F32>(lo, mul, s, r), nv_codes8<DT_F32>(hi, mul, s, r));
            j = u;
        }
        if (n < a.N) reinterpret_cast<uint2*>(a.codes)[(size_t)n * units + u] = c;
        if (FMT == GF_NVFP4 || (g & 1) == 0) a.scales[tiled_index(n, j, a.ktiles)] = n < a.N ? (uint8_t)byte : (uint8_t)0;
    }
    // scales past K in the last tile
    for (int j = a.K / Format<FMT>::kBlock + g; j < a.ktiles * 4; j += 4) a.scales[tiled_index(n, j, a.ktiles)] = 0;
    // the last group of 32 channels also clears the rest of its 128-row tile
    if (n0 + 32 >= a.N)
        for (int r = n0 + 32 + (int)(threadIdx.x >> 2); r < (n0 + 128) / 128 * 128; r += 32)
            for (int j = g; j < a.ktiles * 4; j += 4) a.scales[tiled_index(r, j, a.ktiles)] = 0;
}

template <int DT>
cudaError_t quant_dt(const QuantArgs& a, int fmt, cudaStream_t s) {
    if (fmt == GF_MXFP4) {
        const dim3 grid((a.rows_out + 7) / 8, (a.units_out + 31) / 32);
        return launch_behind(mx_quant_kernel<DT>, grid, dim3(32, 8), 0, 1, s, a);
    } else {
        const int warps = (a.K / kUnit + kKeep<DT> * 32 - 1) / (kKeep<DT> * 32);      // of a row
        const int row = 32 * (warps < kNvThreads / 32 ? warps : kNvThreads / 32), rows = kNvThreads / row;
        return launch_behind(nv_quant_kernel<DT>, (a.rows_out + rows - 1) / rows, dim3(row, rows), 0, 1, s, a);
    }
}

template <int FMT>
cudaError_t dequant_fmt(const DequantArgs& a, int dt, cudaStream_t s) {
    const int n = dt == DT_F32 ? kOut<DT_F32> : kOut<DT_BF16>;
    const dim3 grid((a.M + 7) / 8, (a.K / n + 31) / 32), block(32, 8);
    switch (dt) {
        case DT_F32: return launch_behind(fp4_dequant_kernel<FMT, DT_F32>, grid, block, 0, 1, s, a);
        case DT_F16: return launch_behind(fp4_dequant_kernel<FMT, DT_F16>, grid, block, 0, 1, s, a);
        default: return launch_behind(fp4_dequant_kernel<FMT, DT_BF16>, grid, block, 0, 1, s, a);
    }
}

}  // namespace

size_t fp4_scales_bytes(int rows, int K, int fmt, int layout) {
    const int block = fmt == GF_MXFP4 ? 32 : 16;
    if (layout == SC_ROWS) return (size_t)rows * fp4::scale_pitch(K, block);
    return (size_t)((rows + 127) / 128) * fp4::scale_ktiles(K, block) * 512;
}

cudaError_t launch_fp4_quant(int M, int K, const void* X, int x_dtype, long long ldx, int x_rows, const int32_t* rows,
                             int fmt, int layout, void* codes, void* scales, float* row_scale, cudaStream_t s) {
    const int block = fmt == GF_MXFP4 ? 32 : 16;
    QuantArgs a{};
    a.M = M; a.K = K;
    a.X = X; a.ldx_bytes = ldx * (long long)dt_size(x_dtype);
    a.x_rows = x_rows; a.rows = rows;
    a.layout = layout;
    a.pitch = fp4::scale_pitch(K, block);
    a.ktiles = fp4::scale_ktiles(K, block);
    a.rows_out = layout == SC_ROWS ? M : (M + 127) / 128 * 128;
    a.units_out = (layout == SC_ROWS ? a.pitch : a.ktiles * 4) * (block / kUnit);
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    a.row_scale = row_scale;
    switch (x_dtype) {
        case DT_F32: return quant_dt<DT_F32>(a, fmt, s);
        case DT_F16: return quant_dt<DT_F16>(a, fmt, s);
        default: return quant_dt<DT_BF16>(a, fmt, s);
    }
}

cudaError_t launch_fp4_dequant(int M, int K, int fmt, int layout, const void* codes, const void* scales,
                               const float* row_scale, void* Y, int y_dtype, cudaStream_t s) {
    const int block = fmt == GF_MXFP4 ? 32 : 16;
    DequantArgs a{M, K, layout, fp4::scale_pitch(K, block), fp4::scale_ktiles(K, block), static_cast<const uint8_t*>(codes),
                  static_cast<const uint8_t*>(scales), row_scale, Y};
    return fmt == GF_MXFP4 ? dequant_fmt<GF_MXFP4>(a, y_dtype, s) : dequant_fmt<GF_NVFP4>(a, y_dtype, s);
}

cudaError_t launch_fp4_pack(const float* W, int K, int N, int fmt, void* codes, void* scales, float* row_scale, cudaStream_t s) {
    PackArgs a{W, K, N, fp4::scale_ktiles(K, fmt == GF_MXFP4 ? 32 : 16), static_cast<uint8_t*>(codes),
               static_cast<uint8_t*>(scales), row_scale};
    const int grid = (N + 31) / 32;
    if (fmt == GF_MXFP4) fp4_pack_kernel<GF_MXFP4><<<grid, 128, 0, s>>>(a);
    else fp4_pack_kernel<GF_NVFP4><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace qg
