// The microscaled 4-bit formats: device helpers shared by the quantization and product kernels.
//
// A value is an e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and negatives) times its block's scale:
//   MXFP4  blocks of 32, scale e8m0, 2^(byte - 127), byte 255 = NaN (OCP Microscaling Formats v1.0);
//   NVFP4  blocks of 16, scale e4m3 (byte 0x7f = NaN), times one float32 scale per row.
// Every decision below is exact in float32, so any IEEE evaluation of the definition in
// include/qgemm.h gives the same codes: MXFP4 scales by powers of two only; NVFP4's row scale is a
// power of two, its block scale one correctly rounded quotient, and its codes compare |x| with
// t * s where t * s (3 and 4 significant bits) is exact.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.h"

namespace qg {
namespace fp4 {

template <int FMT>
struct Format {
    static constexpr int kBlock = FMT == GF_MXFP4 ? 32 : 16;
};

// Bytes between two rows of the ROWS scale layout.
__host__ __device__ __forceinline__ int scale_pitch(int K, int block) { return (K / block + 15) / 16 * 16; }
// 512-byte tiles (128 rows x 4 scales) along K of the TILED layout.
__host__ __device__ __forceinline__ int scale_ktiles(int K, int block) { return (K / block + 3) / 4; }
__host__ __device__ __forceinline__ size_t tiled_index(int row, int j, int ktiles) {
    return ((size_t)(row >> 7) * ktiles + (j >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (j & 3);
}

// Eight float32 values as e2m1 codes, the first in the lowest half-byte; to the nearest, ties to the
// even code, saturating at 6.
__device__ __forceinline__ uint32_t pack8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// The values of the eight codes of a word, the lowest half-byte's first.
__device__ __forceinline__ void unpack8(uint32_t w, float* v) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// MXFP4: the scale byte of a block whose largest |x| has these bits: floor(log2) - 2, at least
// 2^-127; an infinity or NaN in the block gives the NaN scale. mul = 2^-(byte - 127).
__device__ __forceinline__ uint32_t mx_scale(uint32_t top_bits, float* mul) {
    const uint32_t e = top_bits >> 23;
    const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
    *mul = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
    return byte;
}
// NVFP4: the row scale 2^ge with ge = floor(log2 max|row|) - 10 in [-116, 117], which brings the
// row's largest value to [2^10, 2^11) and its block scale, a sixth of that, below e4m3's 448;
// 1 for a row of zeros, NaN for a row with an infinity or NaN. mul = 2^-ge (0 for that NaN).
__device__ __forceinline__ float nv_row_scale(uint32_t top_bits, float* mul) {
    const int e = (int)(top_bits >> 23);
    if (top_bits == 0u) return *mul = 1.f;
    if (e == 255) {
        *mul = 0.f;
        return __uint_as_float(0x7FC00000u);
    }
    const int ge = min(max(e - 127 - 10, -116), 117);
    *mul = __uint_as_float((uint32_t)(127 - ge) << 23);
    return __uint_as_float((uint32_t)(127 + ge) << 23);
}
// NVFP4: e4m3 byte of a block scale, and its value.
__device__ __forceinline__ uint32_t nv_scale(uint32_t top_bits, float* s) {
    const float r = __fdiv_rn(__uint_as_float(top_bits), 6.f);
    uint32_t byte, h;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(byte) : "f"(0.f), "f"(r));
    byte &= 0xFFu;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
    *s = __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
    return byte;
}
__device__ __forceinline__ float nv_scale_value(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

}  // namespace fp4
}  // namespace qg
