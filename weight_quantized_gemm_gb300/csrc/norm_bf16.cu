// The step between two blocks with X in bf16.
#include "norm.cuh"

namespace qg {
cudaError_t launch_norm_bf16(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s) {
    return norm::launch_x<DT_BF16>(a, s_dtype, y_dtype, s);
}
}  // namespace qg
