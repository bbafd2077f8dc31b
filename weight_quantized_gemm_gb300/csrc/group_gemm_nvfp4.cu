// The grouped product's kernels for one operand form (a translation unit each, compiled in parallel).
#include "group_gemm.cuh"

namespace qg {

cudaError_t launch_group_gemm_nvfp4(const GroupGemmArgs& a, int fmt, cudaStream_t s) { return gg::launch_form<gg::NV>(a, fmt, s); }

}  // namespace qg
