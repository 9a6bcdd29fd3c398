// The tile kernel's instances for fp32 gradients through the activation and its gate.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_f32_grad_mul(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<1, kGradientMul>(g, grid, stream);
}

}  // namespace mx
