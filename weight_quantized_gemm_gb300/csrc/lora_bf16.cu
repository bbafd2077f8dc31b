// The adapters' products with bf16 operands.
#include "lora_many.cuh"

namespace qg {
cudaError_t launch_lora_bf16(const LoraArgs& a, int y_dtype, cudaStream_t s) { return lora::launch_form<true>(a, y_dtype, s); }
}  // namespace qg
