// The C ABI of include/qgemm.h for 4-bit floating point and mixture-of-experts layers: argument
// checks and size queries. As in qgemm_api.cu, every check runs before the first launch.
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qgemm.h"
#include "experts.h"
#include "group_plan.h"

namespace {

int fail(int code, const char* fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return qg::api_fail(code, text);
}
int done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? QGEMM_OK : fail(QGEMM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
int injected() { return fail(QGEMM_ERR_CUDA, "simulated launch failure (fault injection)"); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// null pointers count as aligned: whether they may be null is checked apart
template <class... P>
bool all_aligned16(P... p) {
    return (aligned16(p) && ...);
}
bool valid_dtype(int d) { return d == QGEMM_F32 || d == QGEMM_F16 || d == QGEMM_BF16; }
bool is_fp4(int fmt) { return fmt == QGEMM_FMT_MXFP4 || fmt == QGEMM_FMT_NVFP4; }
constexpr int kMaxRows = 1 << 30;      // of one call, so that rounding up to a tile stays an int
constexpr int kMaxK = (1 << 30) - 64;  // of a product, so that a 16-bit row's bytes stay an int
bool valid_layout(int l) { return l == QGEMM_SCALES_ROWS || l == QGEMM_SCALES_TILED; }

int check_fp4(int rows, int K, int fmt, const char* name) {
    if (!is_fp4(fmt)) return fail(QGEMM_ERR_ARG, "format %d is not a 4-bit format", fmt);
    if (rows < 0 || K <= 0) return fail(QGEMM_ERR_ARG, "invalid sizes %s=%d K=%d", name, rows, K);
    if (K % 64 != 0) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d is not a multiple of 64", K);
    if (rows > kMaxRows) return fail(QGEMM_ERR_UNSUPPORTED, "%s=%d exceeds %d rows", name, rows, kMaxRows);
    if (K > 8 * 32 * 65535) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d exceeds the launch limit", K);
    return QGEMM_OK;
}

// Checks of both product calls; E experts' weights (1 for the dense product).
int check_product(int M, int E, int K, int N, int fmt, const void* A, const void* As, const float* a_scale, const void* Bp,
                  const void* Bs, const float* b_scale, const float* bias, int act, const void* residual, const void* C,
                  int c_dtype) {
    if (fmt < QGEMM_FMT_F16 || fmt > QGEMM_FMT_NVFP4) return fail(QGEMM_ERR_ARG, "unknown format %d", fmt);
    if (M < 0 || E < 0 || K <= 0 || N < 0) return fail(QGEMM_ERR_ARG, "invalid sizes M=%d E=%d K=%d N=%d", M, E, K, N);
    if (!valid_dtype(c_dtype)) return fail(QGEMM_ERR_ARG, "unknown c_dtype %d", c_dtype);
    if (act < QGEMM_ACT_NONE || act > QGEMM_ACT_SWIGLU) return fail(QGEMM_ERR_ARG, "unknown activation %d", act);
    if (K % 64 != 0) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d is not a multiple of 64", K);
    if (K > kMaxK) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d exceeds %d", K, kMaxK);
    if (act == QGEMM_ACT_SWIGLU && N % 2 != 0)
        return fail(QGEMM_ERR_UNSUPPORTED, "SwiGLU pairs channels: N=%d is odd", N);
    if (M > kMaxRows || N > kMaxRows) return fail(QGEMM_ERR_UNSUPPORTED, "M=%d or N=%d exceeds %d", M, N, kMaxRows);
    if (M == 0 || N == 0 || E == 0) return QGEMM_OK;
    if (!A || !Bp || !C) return fail(QGEMM_ERR_ARG, "null A, Bp or C");
    if (is_fp4(fmt) && (!As || !Bs)) return fail(QGEMM_ERR_ARG, "null block scales");
    if (!all_aligned16(A, As, a_scale, Bp, Bs, b_scale, bias, residual, C))
        return fail(QGEMM_ERR_ALIGN, "A, Bp, C, scales, bias and residual must be 16-byte aligned");
    return QGEMM_OK;
}

int check_tiles(const qg::GroupGemmArgs& a, int fmt) {
    if (qg::gg::countable(a, fmt)) return QGEMM_OK;
    return fail(QGEMM_ERR_UNSUPPORTED, "M=%d K=%d N=%d with %d weights make more tiles than can be counted", a.M, a.K, a.N, a.E);
}

}  // namespace

extern "C" {

size_t qgemm_fp4_codes_bytes(int rows, int K) {
    if (rows < 0 || rows > kMaxRows || K <= 0 || K % 64 != 0) return 0;
    return (size_t)rows * K / 2;
}

size_t qgemm_fp4_scales_bytes(int rows, int K, int fmt, int layout) {
    if (rows < 0 || rows > kMaxRows || K <= 0 || K % 64 != 0 || !is_fp4(fmt) || !valid_layout(layout)) return 0;
    return qg::fp4_scales_bytes(rows, K, fmt, layout);
}

int qgemm_fp4_quant(int M, int K, const void* X, int x_dtype, long long ldx, int x_rows, const int32_t* rows, int fmt,
                    int layout, void* codes, void* scales, float* row_scale, void* stream) {
    const int rc = check_fp4(M, K, fmt, "M");
    if (rc != QGEMM_OK) return rc;
    if (!valid_dtype(x_dtype)) return fail(QGEMM_ERR_ARG, "unknown x_dtype %d", x_dtype);
    if (!valid_layout(layout)) return fail(QGEMM_ERR_ARG, "unknown scale layout %d", layout);
    if (x_rows < 0 || ldx < K) return fail(QGEMM_ERR_ARG, "invalid x_rows=%d or ldx=%lld (K=%d)", x_rows, ldx, K);
    if (!rows && x_rows < M) return fail(QGEMM_ERR_ARG, "x_rows=%d is less than M=%d", x_rows, M);
    if (M == 0) return QGEMM_OK;
    if ((!X && x_rows > 0) || !codes || !scales) return fail(QGEMM_ERR_ARG, "null X, codes or scales");
    if (fmt == QGEMM_FMT_NVFP4 && !row_scale) return fail(QGEMM_ERR_ARG, "null row_scale");
    if (!all_aligned16(X, rows, codes, scales, row_scale))
        return fail(QGEMM_ERR_ALIGN, "X, rows, codes, scales and row_scale must be 16-byte aligned");
    if (ldx * (long long)qg::dt_size(x_dtype) % 16 != 0)
        return fail(QGEMM_ERR_ALIGN, "rows of X must start 16-byte aligned (ldx=%lld)", ldx);
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_fp4_quant(M, K, X, x_dtype, ldx, x_rows, rows, fmt, layout, codes, scales, row_scale,
                                     static_cast<cudaStream_t>(stream)),
                "fp4_quant launch");
}

int qgemm_fp4_dequant(int M, int K, int fmt, int layout, const void* codes, const void* scales, const float* row_scale,
                      void* Y, int y_dtype, void* stream) {
    const int rc = check_fp4(M, K, fmt, "M");
    if (rc != QGEMM_OK) return rc;
    if (!valid_dtype(y_dtype)) return fail(QGEMM_ERR_ARG, "unknown y_dtype %d", y_dtype);
    if (!valid_layout(layout)) return fail(QGEMM_ERR_ARG, "unknown scale layout %d", layout);
    if (M == 0) return QGEMM_OK;
    if (!codes || !scales || !Y) return fail(QGEMM_ERR_ARG, "null codes, scales or Y");
    if (!all_aligned16(codes, scales, row_scale, Y))
        return fail(QGEMM_ERR_ALIGN, "codes, scales, row_scale and Y must be 16-byte aligned");
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_fp4_dequant(M, K, fmt, layout, codes, scales, row_scale, Y, y_dtype,
                                       static_cast<cudaStream_t>(stream)),
                "fp4_dequant launch");
}

int qgemm_fp4_pack(const float* W, int K, int N, int fmt, void* Bp, void* Bs, float* b_scale, void* stream) {
    const int rc = check_fp4(N, K, fmt, "N");
    if (rc != QGEMM_OK) return rc;
    if (N == 0) return QGEMM_OK;
    if (!W || !Bp || !Bs) return fail(QGEMM_ERR_ARG, "null W, Bp or Bs");
    if (fmt == QGEMM_FMT_NVFP4 && !b_scale) return fail(QGEMM_ERR_ARG, "null b_scale");
    if (!all_aligned16(W, Bp, Bs, b_scale))
        return fail(QGEMM_ERR_ALIGN, "W, Bp, Bs and b_scale must be 16-byte aligned");
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_fp4_pack(W, K, N, fmt, Bp, Bs, b_scale, static_cast<cudaStream_t>(stream)), "fp4_pack launch");
}

int qgemm_fp4_run(int M, int K, int N, int fmt, const void* A, const void* As, const float* a_scale, const void* Bp,
                  const void* Bs, const float* b_scale, const float* bias, int act, const void* residual, void* C,
                  int c_dtype, void* stream) {
    if (!is_fp4(fmt)) return fail(QGEMM_ERR_ARG, "format %d is not a 4-bit format", fmt);
    const int rc = check_product(M, 1, K, N, fmt, A, As, a_scale, Bp, Bs, b_scale, bias, act, residual, C, c_dtype);
    if (rc != QGEMM_OK || M == 0 || N == 0) return rc;
    const qg::GroupGemmArgs a{M, 1, K, N, nullptr, A, As, a_scale, Bp, Bs, b_scale, bias, act, residual, C, c_dtype};
    const int tc = check_tiles(a, fmt);
    if (tc != QGEMM_OK) return tc;
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_group_gemm(a, fmt, static_cast<cudaStream_t>(stream)), "fp4_run launch");
}

int qgemm_grouped_run(int T, int E, int K, int N, int fmt, const int32_t* offsets, const void* A, const void* As,
                      const float* a_scale, const void* Bp, const void* Bs, const float* b_scale, const float* bias, int act,
                      void* C, int c_dtype, void* stream) {
    const int rc = check_product(T, E, K, N, fmt, A, As, a_scale, Bp, Bs, b_scale, bias, act, nullptr, C, c_dtype);
    if (rc != QGEMM_OK) return rc;
    if (E > QGEMM_MAX_EXPERTS) return fail(QGEMM_ERR_UNSUPPORTED, "E=%d exceeds %d experts", E, QGEMM_MAX_EXPERTS);
    if (T == 0 || N == 0 || E == 0) return QGEMM_OK;
    if (!offsets) return fail(QGEMM_ERR_ARG, "null offsets");
    if (!aligned16(offsets)) return fail(QGEMM_ERR_ALIGN, "offsets must be 16-byte aligned");
    const qg::GroupGemmArgs a{T, E, K, N, offsets, A, As, a_scale, Bp, Bs, b_scale, bias, act, nullptr, C, c_dtype};
    const int tc = check_tiles(a, fmt);
    if (tc != QGEMM_OK) return tc;
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_group_gemm(a, fmt, static_cast<cudaStream_t>(stream)), "grouped_run launch");
}

// Not part of the ABI: how a product is cut (rows of a tile, blocks that share its K), so that tests can tell
// which form of the kernel a shape takes.
void qg_group_plan(int M, int E, int grouped, int K, int N, int fmt, int* rows, int* split) {
    static const int32_t some = 0;
    const qg::GroupGemmArgs a{M, E, K, N, grouped ? &some : nullptr};
    const qg::gg::Choice c = qg::gg::choose(a, fmt);
    *rows = c.bn;
    *split = c.split;
}

size_t qgemm_moe_route_workspace_bytes(int T, int E, int k) {
    if (T <= 0 || E <= 0 || k <= 0 || k > E || E > QGEMM_MAX_EXPERTS || k > QGEMM_MAX_TOPK) return 0;
    return qg::route_needs_workspace(T) ? (size_t)qg::kRouteBlocks * E * sizeof(int32_t) : 0;
}

int qgemm_moe_route(int T, int E, int k, const void* logits, int dtype, long long ld, int renorm, int32_t* expert,
                    float* weight, int32_t* slot, int32_t* row, int32_t* offsets, void* workspace, size_t workspace_bytes,
                    void* stream) {
    if (T < 0 || E <= 0 || k <= 0 || k > E) return fail(QGEMM_ERR_ARG, "invalid sizes T=%d E=%d k=%d", T, E, k);
    if (!valid_dtype(dtype)) return fail(QGEMM_ERR_ARG, "unknown dtype %d", dtype);
    if (renorm != 0 && renorm != 1) return fail(QGEMM_ERR_ARG, "renorm takes 0 or 1, got %d", renorm);
    if (ld < E) return fail(QGEMM_ERR_ARG, "ld=%lld is less than E=%d", ld, E);
    if (E > QGEMM_MAX_EXPERTS || k > QGEMM_MAX_TOPK)
        return fail(QGEMM_ERR_UNSUPPORTED, "E=%d or k=%d exceeds %d experts or %d choices", E, k, QGEMM_MAX_EXPERTS,
                    QGEMM_MAX_TOPK);
    if ((long long)T * k > 1 << 30) return fail(QGEMM_ERR_UNSUPPORTED, "T * k = %lld exceeds 2^30 pairs", (long long)T * k);
    if (!offsets) return fail(QGEMM_ERR_ARG, "null offsets");
    if (T > 0 && (!logits || !expert || !weight || !slot || !row))
        return fail(QGEMM_ERR_ARG, "null logits, expert, weight, slot or row");
    if (!all_aligned16(logits, expert, weight, slot, row, offsets, workspace))
        return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    const size_t need = qgemm_moe_route_workspace_bytes(T, E, k);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(QGEMM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_moe_route(T, E, k, logits, dtype, ld, renorm, expert, weight, slot, row, offsets, workspace,
                                     static_cast<cudaStream_t>(stream)),
                "moe_route launch");
}

int qgemm_moe_combine(int T, int k, int N, int R, const void* Y, int y_dtype, const int32_t* slot, const float* weight,
                      const void* residual, void* out, int out_dtype, void* stream) {
    if (T < 0 || k < 0 || N < 0 || R < 0) return fail(QGEMM_ERR_ARG, "invalid sizes T=%d k=%d N=%d R=%d", T, k, N, R);
    if (!valid_dtype(y_dtype) || !valid_dtype(out_dtype))
        return fail(QGEMM_ERR_ARG, "unknown dtype (y_dtype %d, out_dtype %d)", y_dtype, out_dtype);
    if ((long long)T * (k > 0 ? k : 1) > kMaxRows)
        return fail(QGEMM_ERR_UNSUPPORTED, "T * k = %lld exceeds 2^30 pairs", (long long)T * (k > 0 ? k : 1));
    if (T == 0 || N == 0) return QGEMM_OK;
    if (!out || (k > 0 && (!slot || !weight)) || (R > 0 && !Y)) return fail(QGEMM_ERR_ARG, "null Y, slot, weight or out");
    if (!all_aligned16(Y, slot, weight, residual, out)) return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (N > 64 * 65535) return fail(QGEMM_ERR_UNSUPPORTED, "N=%d exceeds the launch limit", N);
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_moe_combine(T, k, N, R, Y, y_dtype, slot, weight, residual, out, out_dtype,
                                       static_cast<cudaStream_t>(stream)),
                "moe_combine launch");
}

}  // extern "C"
