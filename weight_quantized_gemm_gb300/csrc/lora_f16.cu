// The adapters' products with f16 operands.
#include "lora_many.cuh"

namespace qg {
cudaError_t launch_lora_f16(const LoraArgs& a, int y_dtype, cudaStream_t s) { return lora::launch_form<false>(a, y_dtype, s); }
}  // namespace qg
