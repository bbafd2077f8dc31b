// Internal launch interface of what stands around the layers (adapters, norms, log probabilities), between the
// C ABI (serve_api.cu) and the kernels.
#pragma once

#include "experts.h"

namespace qg {

constexpr int kMaxLoraAdapters = 1024;

enum NormKind { NORM_RMS = 1, NORM_LAYER = 2 };

struct LoraArgs {
    int M, K, N, L, R;
    const int32_t* row;         // [M]
    const int32_t* offsets;     // [L + 1]
    const void* X;              // [M][ldx]
    long long ldx;
    const void* A;              // [L][R][K]
    const void* B;              // [L][N][R]
    const int32_t* rank;        // [L] or none
    const float* scale;         // [L] or none
    void* Y;                    // [M][ldy]
    long long ldy;
};
cudaError_t launch_lora_group(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets, cudaStream_t s);
// rows of Y that start 16-byte aligned, and rows that need not
cudaError_t launch_lora_f16(const LoraArgs& a, int y_dtype, cudaStream_t s);
cudaError_t launch_lora_bf16(const LoraArgs& a, int y_dtype, cudaStream_t s);
cudaError_t launch_lora_loose_f16(const LoraArgs& a, int y_dtype, cudaStream_t s);
cudaError_t launch_lora_loose_bf16(const LoraArgs& a, int y_dtype, cudaStream_t s);
inline cudaError_t launch_lora(const LoraArgs& a, int dtype, int y_dtype, cudaStream_t s) {
    if (a.ldy % (16 / (long long)dt_size(y_dtype)) == 0)
        return dtype == DT_F16 ? launch_lora_f16(a, y_dtype, s) : launch_lora_bf16(a, y_dtype, s);
    return dtype == DT_F16 ? launch_lora_loose_f16(a, y_dtype, s) : launch_lora_loose_bf16(a, y_dtype, s);
}

struct NormArgs {
    int M, K, kind;
    float eps;
    const void* X;              // [M][ldx]
    long long ldx;
    float x_scale;
    int post;
    const float* post_weight;   // [K] or none
    const void* gate;           // [K] (ldg = 0) or rows ldg apart, or none
    long long ldg;
    const void* residual;       // [M][K] or none
    float r_scale;
    void* S;                    // [M][K] or none
    const float* weight;        // [K] or none
    const float* bias;          // [K] or none
    void* Y;                    // [M][K] or none
};
cudaError_t launch_norm_f32(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s);
cudaError_t launch_norm_f16(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s);
inline cudaError_t launch_norm(const NormArgs& a, int x_dtype, int s_dtype, int y_dtype, cudaStream_t s) {
    return x_dtype == DT_F32 ? launch_norm_f32(a, s_dtype, y_dtype, s)
                             : (x_dtype == DT_F16 ? launch_norm_f16(a, s_dtype, y_dtype, s) : launch_norm_bf16(a, s_dtype, y_dtype, s));
}

cudaError_t launch_logprobs(int T, int V, const void* logits, int dtype, long long ld, float scale, const int32_t* token,
                            float* logprob, float* entropy, int k, int32_t* top, float* top_logprob, cudaStream_t s);

}  // namespace qg
