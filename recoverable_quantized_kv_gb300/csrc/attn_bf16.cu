// The attention kernel for bf16 inputs, plain and biased scores.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_bf16(const AttnArgs &P, int grid, bool bias, cudaStream_t s) {
  return bias ? launch_attn_variant<false, 0, true>(P, grid, s) : launch_attn_variant<false, 0, false>(P, grid, s);
}
}  // namespace qv
