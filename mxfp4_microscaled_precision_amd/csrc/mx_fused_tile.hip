// The tile kernel's instances for bf16 outputs, and the choice between it and
// the kernel of few rows.
#include "mx_fused_tile.h"

namespace mx {

hipError_t launch_tiles_bf16(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  return tile::launch_tiles<0, kForward>(g, grid, stream);
}

static hipError_t fused_tile_launch(FusedArgs g, hipStream_t stream) {
  // at most this many tiles: a ragged group has up to two more than its rows'
  int64_t rt = ((int64_t)g.M + tile::kBM - 1) / tile::kBM;
  if (g.kind == MX_K_WGRAD)
    rt *= g.groups;
  else if (g.ends)
    rt = g.rows / tile::kBM + 2 * (int64_t)std::min(g.groups, g.rows);
  // a group's columns may begin at any row of B
  const int64_t cols =
      (int64_t)g.N + (g.kind == MX_K_FPROP && g.groups > 1 && g.N % 64 != 0 ? 63 : 0);
  g.col_tiles = (int)((cols + tile::kBN - 1) / tile::kBN);
  g.by_col_tiles = DivideBy((uint32_t)g.col_tiles);
  g.by_row_tiles = DivideBy((uint32_t)((g.M + tile::kBM - 1) / tile::kBM));
  const int64_t tiles = rt * g.col_tiles;
  if (tiles == 0) return hipSuccess;
  if (tiles > INT32_MAX / 2 || g.groups > tile::kTileGroups) return hipErrorInvalidValue;
  const dim3 grid((unsigned)std::min<int64_t>(2 * tiles, cu_count()));
  if (g.grad && g.e.mul)
    return g.out_bf16 ? launch_tiles_bf16_grad_mul(g, grid, stream)
                      : launch_tiles_f32_grad_mul(g, grid, stream);
  if (g.grad)
    return g.out_bf16 ? launch_tiles_bf16_grad(g, grid, stream)
                      : launch_tiles_f32_grad(g, grid, stream);
  if (g.e.mul && g.e.residual)
    return g.out_bf16 ? launch_tiles_bf16_both(g, grid, stream)
                      : launch_tiles_f32_both(g, grid, stream);
  return g.out_bf16 ? launch_tiles_bf16(g, grid, stream) : launch_tiles_f32(g, grid, stream);
}

// The kernel of few rows where its 64x64 tiles (about one more per group than its
// rows fill) go round the compute units three times at most: a 256-wide tile's stages
// and epilogue then take longer than all of them. Where the columns do not end at a
// multiple of 64 it is taken up to 160 GFLOP: the tile kernel's last columns are a wave's
// that reads and writes them one by one. And where a group has a handful of rows on
// average: what counts is then that its weights are read once. Measured, us (few rows /
// tiles): with SiLU, 512x4096x4096 16.6 / 22.4, 128x14336x4096 15.6 / 23.5,
// 2048x1024x4096 12.1 / 21.9, and past the limit 1024x4096x4096 25.8 / 23.3,
// 256x14336x4096 26.7 / 23.4 (the plain product alone: 14.4
// and 15.0); 256 rows of 8 experts 4096x4096 25.2 / 29.7, of 64
// experts 2048x1024 18.3 / 21.5, 4096 rows of those 45.7 / 27.6; bf16 with a
// residual that ends inside 64 columns, 7417x3324x160 52 / 162 (with bias and SiLU as
// well 64 / 200), 4096x4097x4096 78 / 182,
// 8192x1056x4096 50 / 95 and without one 8192x8200x2048 (275 GFLOP) 187 / 156.
hipError_t fused_launch(const FusedArgs &g, hipStream_t stream) {
  const bool wgrad = g.kind == MX_K_WGRAD;
  const int64_t rows = wgrad ? (int64_t)g.groups * ((g.M + 63) / 64)
                             : (g.rows + 63) / 64 + (g.ends ? std::min(g.groups, g.rows) : 0);
  const bool few = rows * (((int64_t)g.N + 63) / 64) <= 3 * (int64_t)cu_count();
  const double flops = 2.0 * g.N * (wgrad ? g.M : g.rows) * (wgrad ? g.rows : 128.0 * g.a_slices);
  const bool ragged = (g.N % 64 != 0 || !g.e.vec) && flops <= 160e9;
  const bool handful = !wgrad && g.rows / g.groups <= 8;
  return few || ragged || handful || g.groups > tile::kTileGroups ? fused_small_launch(g, stream)
                                                                  : fused_tile_launch(g, stream);
}

}  // namespace mx
