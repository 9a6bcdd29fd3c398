// The tile kernel's instances for bf16 outputs, and the choice between it and
// the kernel of few rows.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_bf16(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<0, false>(g, grid, stream);
}

static hipError_t fused_tile_launch(const FusedArgs &g, hipStream_t stream) {
  // at most this many tiles: a ragged group has up to two more than its rows'
  int64_t rt = ((int64_t)g.M + tile::kBM - 1) / tile::kBM;
  if (g.kind == MX_K_WGRAD)
    rt *= g.groups;
  else if (g.ends)
    rt = g.rows / tile::kBM + 2 * (int64_t)std::min(g.groups, g.rows);
  const int64_t tiles = rt * ((g.N + 63 + tile::kBN - 1) / tile::kBN);
  if (tiles == 0) return hipSuccess;
  if (tiles > INT32_MAX / 2 || g.groups > tile::kTileGroups) return hipErrorInvalidValue;
  const dim3 grid((unsigned)std::min<int64_t>(2 * tiles, cu_count()));
  if (g.grad)
    return g.out_bf16 ? launch_tiles_bf16_grad(g, grid, stream)
                      : launch_tiles_f32_grad(g, grid, stream);
  return g.out_bf16 ? launch_tiles_bf16(g, grid, stream) : launch_tiles_f32(g, grid, stream);
}

hipError_t fused_launch(const FusedArgs &g, hipStream_t stream) {
  const int64_t rows = g.kind == MX_K_WGRAD ? g.M : g.rows / g.groups;   // of a group, on average
  return g.groups > tile::kTileGroups || rows <= 64 ? fused_small_launch(g, stream)
                                              : fused_tile_launch(g, stream);
}

}  // namespace mx
