// The grouped product's kernels for one operand form (a translation unit each, compiled in parallel).
#include "group_gemm.cuh"

namespace qg {

cudaError_t launch_group_gemm_mxfp4(const GroupGemmArgs& a, int fmt, cudaStream_t s) { return gg::launch_form<gg::MX>(a, fmt, s); }

}  // namespace qg
