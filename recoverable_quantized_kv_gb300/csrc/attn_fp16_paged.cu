// The attention kernel for fp16 inputs over a cache in pages, plain and biased scores.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_fp16_paged(const AttnArgs &P, int grid, bool bias, cudaStream_t s) {
  return bias ? launch_attn_variant<true, 0, true, true>(P, grid, s) : launch_attn_variant<true, 0, false, true>(P, grid, s);
}
}  // namespace qv
