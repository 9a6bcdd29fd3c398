// The tile kernel's instances for bf16 outputs with a gate and a residual.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_bf16_both(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<0, kForwardBoth>(g, grid, stream);
}

}  // namespace mx
