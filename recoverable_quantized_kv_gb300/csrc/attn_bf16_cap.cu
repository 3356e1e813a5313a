// The attention kernel for bf16 inputs, capped scores.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_bf16_cap(const AttnArgs &P, int grid, bool bias, cudaStream_t s) {
  return bias ? launch_attn_variant<false, 1, true>(P, grid, s) : launch_attn_variant<false, 1, false>(P, grid, s);
}
}  // namespace qv
