// The tile kernel's instances for fp32 outputs.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_f32(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<1, kForward>(g, grid, stream);
}

}  // namespace mx
