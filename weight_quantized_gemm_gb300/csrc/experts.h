// Internal launch interface of the 4-bit floating-point and mixture-of-experts calls, between their C
// ABI (experts_api.cu) and kernels.
#pragma once

#include "internal.h"

namespace qg {

// Operand formats of the 4-bit floating-point and grouped products, and the layouts of their block
// scales (the C ABI's QGEMM_FMT_* and QGEMM_SCALES_* values).
enum GroupFmt { GF_F16 = 1, GF_BF16 = 2, GF_MXFP4 = 3, GF_NVFP4 = 4 };
enum ScaleLayout { SC_ROWS = 0, SC_TILED = 1 };
// The activation after internal.h's Act that these products have alone (channel pairs to one output).
constexpr int ACT_SWIGLU = 4;

// Counts a compute call towards QGEMM_OPT_FAULT_INJECT; true for the call that is to fail.
bool api_inject_fault();

// Launches a kernel that may come up behind the one before it in the stream (it calls grid_wait
// before it touches memory); cluster: blocks of a thread-block cluster.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, unsigned cluster, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

size_t fp4_scales_bytes(int rows, int K, int fmt, int layout);
cudaError_t launch_fp4_quant(int M, int K, const void* X, int x_dtype, long long ldx, int x_rows, const int32_t* rows,
                             int fmt, int layout, void* codes, void* scales, float* row_scale, cudaStream_t s);
cudaError_t launch_fp4_dequant(int M, int K, int fmt, int layout, const void* codes, const void* scales,
                               const float* row_scale, void* Y, int y_dtype, cudaStream_t s);
cudaError_t launch_fp4_pack(const float* W, int K, int N, int fmt, void* codes, void* scales, float* row_scale,
                            cudaStream_t s);
struct GroupGemmArgs {
    int M, E, K, N;             // M rows in all; E experts (1 for a dense product)
    const int32_t* offsets;     // [E + 1] first row of each expert, or none: all rows are expert 0's
    const void* A;
    const void* As;             // block scales, ROWS layout (4-bit formats)
    const float* a_scale;       // [M] or none
    const void* B;              // [E][N][K]
    const void* Bs;             // [E] x TILED layout
    const float* b_scale;       // [E][N] or none
    const float* bias;          // [E][N] or none
    int act;
    const void* residual;       // C's type and shape, or none
    void* C;
    int c_dtype;
};
cudaError_t launch_group_gemm_half(const GroupGemmArgs& a, int fmt, cudaStream_t s);
cudaError_t launch_group_gemm_mxfp4(const GroupGemmArgs& a, int fmt, cudaStream_t s);
cudaError_t launch_group_gemm_nvfp4(const GroupGemmArgs& a, int fmt, cudaStream_t s);
inline cudaError_t launch_group_gemm(const GroupGemmArgs& a, int fmt, cudaStream_t s) {
    return fmt == GF_MXFP4 ? launch_group_gemm_mxfp4(a, fmt, s)
                           : (fmt == GF_NVFP4 ? launch_group_gemm_nvfp4(a, fmt, s) : launch_group_gemm_half(a, fmt, s));
}
// The router's launches: up to kRouteSmallTokens tokens in one thread block, else kRouteBlocks blocks
// at most, with a histogram of E counts each in the workspace.
constexpr int kRouteSmallTokens = 32;
constexpr int kRouteBlocks = kTargetSms;
inline bool route_needs_workspace(int T) { return T > kRouteSmallTokens; }
cudaError_t launch_moe_route(int T, int E, int k, const void* logits, int dtype, long long ld, int renorm, int32_t* expert,
                             float* weight, int32_t* slot, int32_t* row, int32_t* offsets, void* workspace, cudaStream_t s);
cudaError_t launch_moe_combine(int T, int k, int N, int R, const void* Y, int y_dtype, const int32_t* slot,
                               const float* weight, const void* residual, void* out, int out_dtype, cudaStream_t s);

}  // namespace qg
