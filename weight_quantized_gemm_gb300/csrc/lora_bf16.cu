// The adapters' products with bf16 operands, rows of Y 16-byte aligned.
#include "lora_many.cuh"

namespace qg {
cudaError_t launch_lora_bf16(const LoraArgs& a, int y_dtype, cudaStream_t s) { return lora::launch_form<true, true>(a, y_dtype, s); }
}  // namespace qg
