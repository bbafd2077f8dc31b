// The C ABI of include/qgemm.h for what stands around the layers: argument checks. As in qgemm_api.cu, every
// check runs before the first launch.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qgemm.h"
#include "serve.h"

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
static_assert(QGEMM_MAX_ADAPTERS == qg::kMaxLoraAdapters, "how many the search for a tile takes");
constexpr int kMax = 1 << 30;      // rows and columns of one call, so that rounding up to a tile stays an int
// rows `ld` values apart start 16-byte aligned (of any size: the product is not formed)
bool row_aligned(long long ld, int dtype) { return ld % (16 / (long long)qg::dt_size(dtype)) == 0; }
// the last of `rows` rows starts within 2^62 bytes
bool reachable(int rows, long long ld) { return rows == 0 || ld <= (1LL << 60) / rows; }

}  // namespace

extern "C" {

int qgemm_lora_group(int M, int L, const int32_t* adapter, int32_t* row, int32_t* offsets, void* stream) {
    if (M < 0 || L <= 0) return fail(QGEMM_ERR_ARG, "invalid sizes M=%d L=%d", M, L);
    if (L > QGEMM_MAX_ADAPTERS) return fail(QGEMM_ERR_UNSUPPORTED, "L=%d exceeds %d adapters", L, QGEMM_MAX_ADAPTERS);
    if (M > kMax) return fail(QGEMM_ERR_UNSUPPORTED, "M=%d exceeds %d rows", M, kMax);
    if (!offsets || (M > 0 && (!adapter || !row))) return fail(QGEMM_ERR_ARG, "null adapter, row or offsets");
    if (!all_aligned16(adapter, row, offsets)) return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_lora_group(M, L, adapter, row, offsets, static_cast<cudaStream_t>(stream)), "lora_group launch");
}

int qgemm_lora_run(int M, int K, int N, int L, int R, int dtype, const int32_t* row, const int32_t* offsets, const void* X,
                   long long ldx, const void* A, const void* B, const int32_t* rank, const float* scale, void* Y,
                   int y_dtype, long long ldy, void* stream) {
    if (M < 0 || K <= 0 || N < 0 || L <= 0 || R <= 0)
        return fail(QGEMM_ERR_ARG, "invalid sizes M=%d K=%d N=%d L=%d R=%d", M, K, N, L, R);
    if (dtype != QGEMM_F16 && dtype != QGEMM_BF16) return fail(QGEMM_ERR_ARG, "dtype %d is not f16 or bf16", dtype);
    if (!valid_dtype(y_dtype)) return fail(QGEMM_ERR_ARG, "unknown y_dtype %d", y_dtype);
    if (ldx < K || ldy < N) return fail(QGEMM_ERR_ARG, "ldx=%lld is less than K=%d, or ldy=%lld less than N=%d", ldx, K, ldy, N);
    if (K % 64 != 0) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d is not a multiple of 64", K);
    if (R % 8 != 0 || R > QGEMM_MAX_RANK)
        return fail(QGEMM_ERR_UNSUPPORTED, "R=%d is not a multiple of 8 up to %d", R, QGEMM_MAX_RANK);
    if (L > QGEMM_MAX_ADAPTERS) return fail(QGEMM_ERR_UNSUPPORTED, "L=%d exceeds %d adapters", L, QGEMM_MAX_ADAPTERS);
    if (M > kMax || K > kMax || N > kMax) return fail(QGEMM_ERR_UNSUPPORTED, "M=%d, K=%d or N=%d exceeds %d", M, K, N, kMax);
    if (!reachable(M, ldx) || !reachable(M, ldy)) return fail(QGEMM_ERR_UNSUPPORTED, "ldx=%lld or ldy=%lld is too large", ldx, ldy);
    if (M == 0 || N == 0) return QGEMM_OK;
    if (!row || !offsets || !X || !A || !B || !Y) return fail(QGEMM_ERR_ARG, "null row, offsets, X, A, B or Y");
    if (!all_aligned16(row, offsets, X, A, B, rank, scale, Y)) return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (!row_aligned(ldx, dtype)) return fail(QGEMM_ERR_ALIGN, "rows of X must start 16-byte aligned (ldx=%lld)", ldx);
    if (qg::api_inject_fault()) return injected();
    const qg::LoraArgs a{M, K, N, L, R, row, offsets, X, ldx, A, B, rank, scale, Y, ldy};
    return done(qg::launch_lora(a, dtype, y_dtype, static_cast<cudaStream_t>(stream)), "lora_run launch");
}

int qgemm_norm_run(int M, int K, int kind, float eps, const void* X, int x_dtype, long long ldx, float x_scale, int post,
                   const float* post_weight, const void* gate, long long ldg, const void* residual, float r_scale, void* S,
                   int s_dtype, const float* weight, const float* bias, void* Y, int y_dtype, void* stream) {
    if (M < 0 || K <= 0) return fail(QGEMM_ERR_ARG, "invalid sizes M=%d K=%d", M, K);
    if (kind != QGEMM_NORM_RMS && kind != QGEMM_NORM_LAYER) return fail(QGEMM_ERR_ARG, "unknown norm %d", kind);
    if (!(eps >= 0.f) || isinf(eps)) return fail(QGEMM_ERR_ARG, "eps must be finite and not negative");
    if (!valid_dtype(x_dtype) || !valid_dtype(s_dtype) || !valid_dtype(y_dtype))
        return fail(QGEMM_ERR_ARG, "unknown dtype (x_dtype %d, s_dtype %d, y_dtype %d)", x_dtype, s_dtype, y_dtype);
    if (post != 0 && post != 1) return fail(QGEMM_ERR_ARG, "post takes 0 or 1, got %d", post);
    if (!post && post_weight) return fail(QGEMM_ERR_ARG, "post_weight without post");
    if (ldx < K || (gate && ldg != 0 && ldg < K)) return fail(QGEMM_ERR_ARG, "ldx=%lld or ldg=%lld is less than K=%d", ldx, ldg, K);
    if (K % 64 != 0) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d is not a multiple of 64", K);
    if (K > QGEMM_MAX_NORM_K) return fail(QGEMM_ERR_UNSUPPORTED, "K=%d exceeds %d", K, QGEMM_MAX_NORM_K);
    if (M > kMax) return fail(QGEMM_ERR_UNSUPPORTED, "M=%d exceeds %d rows", M, kMax);
    if (!reachable(M, ldx) || (gate && !reachable(M, ldg)))
        return fail(QGEMM_ERR_UNSUPPORTED, "ldx=%lld or ldg=%lld is too large", ldx, ldg);
    if (M == 0) return QGEMM_OK;
    if (!X || (!S && !Y)) return fail(QGEMM_ERR_ARG, "null X, or neither S nor Y");
    if (!all_aligned16(X, post_weight, gate, residual, S, weight, bias, Y))
        return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (!row_aligned(ldx, x_dtype) || (gate && !row_aligned(ldg, x_dtype)))
        return fail(QGEMM_ERR_ALIGN, "rows of X and gate must start 16-byte aligned (ldx=%lld, ldg=%lld)", ldx, ldg);
    if (Y == X && (y_dtype != x_dtype || ldx != K)) return fail(QGEMM_ERR_ARG, "Y may be X only with its type and ldx = K");
    if (qg::api_inject_fault()) return injected();
    const qg::NormArgs a{M, K, kind, eps, X, ldx, x_scale, post, post_weight, gate, ldg, residual, r_scale, S, weight, bias, Y};
    return done(qg::launch_norm(a, x_dtype, s_dtype, y_dtype, static_cast<cudaStream_t>(stream)), "norm_run launch");
}

int qgemm_logprobs(int T, int V, const void* logits, int dtype, long long ld, float scale, const int32_t* token,
                   float* logprob, float* entropy, int k, int32_t* top, float* top_logprob, void* stream) {
    if (T < 0 || V <= 0 || k < 0) return fail(QGEMM_ERR_ARG, "invalid sizes T=%d V=%d k=%d", T, V, k);
    if (!valid_dtype(dtype)) return fail(QGEMM_ERR_ARG, "unknown dtype %d", dtype);
    if (ld < V) return fail(QGEMM_ERR_ARG, "ld=%lld is less than V=%d", ld, V);
    if (!(scale > 0.f) || isinf(scale)) return fail(QGEMM_ERR_ARG, "scale must be finite and above 0");
    if (k > QGEMM_MAX_TOPK) return fail(QGEMM_ERR_UNSUPPORTED, "k=%d exceeds %d", k, QGEMM_MAX_TOPK);
    if (T > kMax || V > kMax) return fail(QGEMM_ERR_UNSUPPORTED, "T=%d or V=%d exceeds %d", T, V, kMax);
    if (!reachable(T, ld)) return fail(QGEMM_ERR_UNSUPPORTED, "ld=%lld is too large", ld);
    if (T == 0) return QGEMM_OK;
    if (!logits || (!token != !logprob) || (k > 0 && (!top || !top_logprob)))
        return fail(QGEMM_ERR_ARG, "null logits, top or top_logprob, or token without logprob");
    if (!all_aligned16(logits, token, logprob, entropy, top, top_logprob))
        return fail(QGEMM_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (!logprob && !entropy && k == 0) return QGEMM_OK;
    if (qg::api_inject_fault()) return injected();
    return done(qg::launch_logprobs(T, V, logits, dtype, ld, scale, token, logprob, entropy, k, top, top_logprob,
                                    static_cast<cudaStream_t>(stream)),
                "logprobs launch");
}

}  // extern "C"
