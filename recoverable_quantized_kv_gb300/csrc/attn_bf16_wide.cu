// The attention kernel for bf16 inputs, scores with a wide cap.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_bf16_wide(const AttnArgs &P, int grid, bool bias, cudaStream_t s) {
  return bias ? launch_attn_variant<false, 2, true>(P, grid, s) : launch_attn_variant<false, 2, false>(P, grid, s);
}
}  // namespace qv
