// The tile kernel's instances for bf16 gradients through the activation and its gate.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_bf16_grad_mul(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<0, kGradientMul>(g, grid, stream);
}

}  // namespace mx
