// The adapters' products with f16 operands, rows of Y that start at any value.
#include "lora_many.cuh"

namespace qg {
cudaError_t launch_lora_loose_f16(const LoraArgs& a, int y_dtype, cudaStream_t s) { return lora::launch_form<false, false>(a, y_dtype, s); }
}  // namespace qg
