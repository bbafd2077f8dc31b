// The step between two blocks with X in f32.
#include "norm.cuh"

namespace qg {
cudaError_t launch_norm_f32(const NormArgs& a, int s_dtype, int y_dtype, cudaStream_t s) {
    return norm::launch_x<DT_F32>(a, s_dtype, y_dtype, s);
}
}  // namespace qg
