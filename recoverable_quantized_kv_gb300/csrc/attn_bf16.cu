// The attention kernel for bf16 inputs.
#include "attn_dev.cuh"

namespace qv {
cudaError_t launch_attn_bf16(const AttnArgs &P, int grid, bool cap, bool bias, cudaStream_t s) {
  return launch_attn_type<false>(P, grid, cap, bias, s);
}
}  // namespace qv
