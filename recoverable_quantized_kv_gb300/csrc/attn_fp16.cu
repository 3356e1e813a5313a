// The attention kernel for fp16 inputs.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_fp16(const AttnArgs &P, int grid, bool cap, bool bias, cudaStream_t s) {
  return launch_attn_type<true>(P, grid, cap, bias, s);
}
}  // namespace qv
