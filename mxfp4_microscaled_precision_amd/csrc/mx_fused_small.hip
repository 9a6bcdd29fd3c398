// Products with an epilogue and products grouped by expert, where there are
// few rows: MXFP4 operands in the packed tile layout (see mxfp4.h), fp32 sums.
//
// With few rows a product is bound by reading the weights once, and a 256-wide
// tile per compute unit would leave most of the card idle. Here a workgroup
// takes 64 or 16 columns of 64 or 16 rows and splits the reduction over its waves:
// wave w reads slices w, w + W, .. straight from memory into registers (a
// tile of the layout is one contiguous 1 KB load of 16 bytes per lane, which
// is the matrix instruction's fragment), and the waves' sums meet in LDS,
// added in wave order, before the epilogue.
//
// Bound by the weights' bytes where they are many, by latency elsewhere: one row
// of 14336x4096 weights (31 MB) takes 6.7 us, 48 rows of 8 experts 4096x4096
// (71 MB) 14.7 us, 4.9 TB/s; 1237x2081x2080 in fp32 with bias, GELU and residual
// 20 us, 777x1056x992's gradient 7.5 us. Of more than some 64 rows it is bound by
// this tiling: the operands are asked for once per 64x64 tile (93 MB for the first of
// these, whose operands are 3.7 MB), two slices at a time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx_epilogue.h"
#include "mx_gemm_common.h"
#include "mx_groups.h"
#include "mx_kernels.h"

namespace mx {

namespace {

using namespace gemm;

// What a wave reads of one 128-deep slice: R row groups of A, J of B (four or
// one), and the scales of the four row groups that each sits among.
template <int R, int J>
struct Slice {
  uint4 a[R], b[J];
  uint32_t sa, sb;
};

template <int R, int J, int kWaves, int F32, bool GRAD>
__global__ __launch_bounds__(64 * kWaves) void fused_small_kernel(FusedArgs g, int row_tiles) {
  constexpr int kRows = 16 * R, kCols = 16 * J;
  constexpr int kPitch = kCols + 4;                // LDS row of fp32 sums, 16 bytes of padding
  __shared__ __attribute__((aligned(16))) float red[kWaves][kRows][kPitch];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int rt = (int)(blockIdx.x % (unsigned)row_tiles), ct = (int)(blockIdx.x / (unsigned)row_tiles);

  // the tile: A rows from ra on (C rows c_row + them, those in [first, last)),
  // B rows from rb on (C columns col0 ..), nk slices from ka and kb on
  int e = 0, ra, first = 0, last = g.M, ka = 0, kb = 0, nk = g.a_slices, rb = ct * kCols, col0 = rb;
  int64_t c_row = 0;
  if (g.kind == MX_K_WGRAD) {
    const int tm = (g.M + kRows - 1) / kRows;
    e = rt / tm;
    ra = (rt - e * tm) * kRows;
    c_row = (int64_t)e * g.M;
    const Group gr = find_group<false>(g.ends, g.groups, g.rows, 0, e, CountSlices());
    ka = kb = gr.before;
    nk = CountSlices()(gr.first, gr.last);
  } else if (g.ends == nullptr) {
    ra = rt * kRows;
  } else {
    const Group gr =
        find_group<true>(g.ends, g.groups, g.rows, 0, rt, CountTiles<kRows, kRows>());
    if (gr.g == g.groups) return;
    e = gr.g;
    first = gr.first;
    last = gr.last;
    ra = (first & ~(kRows - 1)) + (rt - gr.before) * kRows;
    if (g.kind == MX_K_DGRAD) {
      kb = e * g.a_slices;
    } else {
      const int64_t at = (int64_t)e * g.N;         // group e's first row of B
      rb = (int)(at & ~(int64_t)(kCols - 1)) + ct * kCols;
      col0 = (int)(rb - at);
    }
  }
  if (col0 >= g.N) return;

  v4f acc[R][J];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int ga = ra >> 4, gb = rb >> 4;
  const uint8_t *pa = g.a_codes + ((int64_t)ga * g.a_slices + ka) * 1024 + lane * 16;
  const uint8_t *pb = g.b_codes + ((int64_t)gb * g.b_slices + kb) * 1024 + lane * 16;
  const uint8_t *qa = g.a_scales + ((int64_t)ka * g.a_panels + (ga >> 4)) * 1024 +
                      ((ga >> 2) & 3) * 256 + lane * 4;
  const uint8_t *qb = g.b_scales + ((int64_t)kb * g.b_panels + (gb >> 4)) * 1024 +
                      ((gb >> 2) & 3) * 256 + lane * 4;
  auto read = [&](Slice<R, J> &s, int k) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      s.b[j] = *reinterpret_cast<const uint4 *>(pb + ((int64_t)j * g.b_slices + k) * 1024);
#pragma unroll
    for (int i = 0; i < R; ++i)
      s.a[i] = *reinterpret_cast<const uint4 *>(pa + ((int64_t)i * g.a_slices + k) * 1024);
    s.sb = *reinterpret_cast<const uint32_t *>(qb + (int64_t)k * g.b_panels * 1024);
    s.sa = *reinterpret_cast<const uint32_t *>(qa + (int64_t)k * g.a_panels * 1024);
  };
  auto multiply = [&](const Slice<R, J> &s) {
    // one row group: its byte of the four comes to the front
    const uint32_t sa = R == 1 ? s.sa >> (8 * (ga & 3)) : s.sa;
    const uint32_t sb = J == 1 ? s.sb >> (8 * (gb & 3)) : s.sb;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // (the byte selects are part of the instruction)
#define MX_TILE(I, K)                                                                  \
  if constexpr (K < J)                                                                 \
    if (i == I) acc[i][K] = mfma_fp4<K, I>(s.b[K], s.a[i], acc[i][K], sb, sa);
#define MX_ROW(I) MX_TILE(I, 0) MX_TILE(I, 1) MX_TILE(I, 2) MX_TILE(I, 3)
      MX_ROW(0) MX_ROW(1) MX_ROW(2) MX_ROW(3)
#undef MX_ROW
#undef MX_TILE
    }
  };
  // two slices ahead of the one that is multiplied
  Slice<R, J> s0, s1;
  int k = wave;
  if (k < nk) read(s0, k);
  for (; k < nk; k += 2 * kWaves) {
    if (k + kWaves < nk) read(s1, k + kWaves);
    multiply(s0);
    if (k + kWaves < nk) {
      if (k + 2 * kWaves < nk) read(s0, k + 2 * kWaves);
      multiply(s1);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j)
      *reinterpret_cast<v4f *>(&red[wave][16 * i + lr][16 * j + 4 * lg]) = acc[i][j];

  // A lane has eight columns of a row where the workgroup's columns are all the
  // matrix's (and its rows less than 16 MB apart); else one column of four rows, so
  // that the lanes still access adjacent columns.
  const bool vec = g.e.vec && col0 >= 0 && col0 + kCols <= g.N;
  if (vec) {
    constexpr int kUnits = kCols / 8, kStep = 64 / kUnits;        // rows of a wave at a time
    __syncthreads();
#pragma unroll 1
    for (int r8 = wave * kStep; r8 < kRows; r8 += kStep * kWaves) {
      const int r = r8 + lane / kUnits, c8 = lane % kUnits * 8, row = ra + r, col = col0 + c8;
      if (r >= kRows || row < first || row >= last) continue;
      const int64_t at = c_row + row;
      Row8<F32> mul, other, c, second;
      if (g.e.mul) mul = load_row8<F32>(g.e.mul, at * g.e.ldmul + col);
      if (other_of<GRAD>(g.e)) other = load_row8<F32>(other_of<GRAD>(g.e), at * other_ld<GRAD>(g.e) + col);
      float v[8], bias[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0.0f;
        bias[i] = !GRAD && g.e.bias ? load_bias(g.e, (int64_t)e * g.N + col + i) : 0.0f;
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f d = *reinterpret_cast<const v4f *>(&red[w][r][c8 + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * h + i] += d[i];
        }
      }
      with_act(g.e.act, [&](auto act) {
        epilogue8<F32, GRAD, act()>(v, bias, g.e.mul, g.e.residual, mul, other, c, second);
      });
      if (second_of<GRAD>(g.e)) store_row8<F32>(second_of<GRAD>(g.e), at * second_ld<GRAD>(g.e) + col, second);
      store_row8<F32>(g.c, at * g.ldc + col, c);
    }
    return;
  }
  const int mine = lane % kCols, col = col0 + mine;
  const bool in = col >= 0 && col < g.N;
  const float bias = !GRAD && g.e.bias && in ? load_bias(g.e, (int64_t)e * g.N + col) : 0.0f;
  __syncthreads();
  if (!in) return;
#pragma unroll 1
  for (int r4 = (wave * (64 / kCols) + lane / kCols) * 4; r4 < kRows;
       r4 += 4 * (64 / kCols) * kWaves) {
    float v[4], m[4], o[4], a[4], b[4];
    const void *const from = other_of<GRAD>(g.e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = ra + r4 + i;
      const bool mine = row >= first && row < last;
      m[i] = mine && g.e.mul ? load_one<F32>(g.e.mul, (c_row + row) * g.e.ldmul + col) : 0.0f;
      o[i] = mine && from ? load_one<F32>(from, (c_row + row) * other_ld<GRAD>(g.e) + col) : 0.0f;
      v[i] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += red[w][r4 + i][mine];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bias;
    with_act(g.e.act, [&](auto act) {
      auto mul = [&](int k) { return m[k]; };
      auto other = [&](int k) { return o[k]; };
      if (GRAD && !g.e.mul)
        epilogue_of<kGradient, act()>(v, mul, other, false, false, a, b);
      else
        epilogue_of<GRAD ? kGradientMul : kForwardBoth, act()>(v, mul, other, g.e.mul,
                                                               g.e.residual, a, b);
    });
    void *const to2 = second_of<GRAD>(g.e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = ra + r4 + i;
      if (row < first || row >= last) continue;
      if (to2) store_one<F32>(to2, (c_row + row) * second_ld<GRAD>(g.e) + col, b[i]);
      store_one<F32>(g.c, (c_row + row) * g.ldc + col, a[i]);
    }
  }
}

// Tiles of `rows` rows and of `cols` columns, at most.
int64_t count_row_tiles(const FusedArgs &g, int rows) {
  const int64_t tm = ((int64_t)g.M + rows - 1) / rows;
  if (g.kind == MX_K_WGRAD) return tm * g.groups;
  // a group's tiles begin at a multiple of `rows`: up to two more than its rows'
  return g.ends ? g.rows / rows + 2 * (int64_t)std::min(g.groups, g.rows) : tm;
}

int64_t count_col_tiles(const FusedArgs &g, int cols) {
  const int64_t ct = ((int64_t)g.N + cols - 1) / cols;
  return ct + (g.kind == MX_K_FPROP && g.groups > 1 && g.N % cols ? 1 : 0);   // any first column
}

template <int R, int J, int W, int F32, bool GRAD>
hipError_t launch_small(const FusedArgs &g, hipStream_t stream) {
  const int64_t rt = count_row_tiles(g, 16 * R), ct = count_col_tiles(g, 16 * J);
  if (rt * ct == 0) return hipSuccess;
  if (rt * ct > INT32_MAX) return hipErrorInvalidValue;
  return launch(fused_small_kernel<R, J, W, F32, GRAD>, dim3((unsigned)(rt * ct)), dim3(64 * W), 0,
                stream, g, (int)rt);
}

template <int R, int J, int W>
hipError_t launch_tile(const FusedArgs &g, hipStream_t stream) {
  if (g.grad)
    return g.out_bf16 ? launch_small<R, J, W, 0, true>(g, stream)
                      : launch_small<R, J, W, 1, true>(g, stream);
  return g.out_bf16 ? launch_small<R, J, W, 0, false>(g, stream)
                    : launch_small<R, J, W, 1, false>(g, stream);
}

}  // namespace

hipError_t fused_small_launch(const FusedArgs &g, hipStream_t stream) {
  const int64_t cus = cu_count();
  const int rows = g.kind == MX_K_WGRAD ? g.M : g.rows / g.groups;   // of a group, on average
  // workgroups of 64 columns on less than half of the card: 16 columns each
  const int64_t tiles = count_row_tiles(g, rows <= 16 ? 16 : 64) * count_col_tiles(g, 64);
  if (rows <= 16)
    return 2 * tiles <= cus ? launch_tile<1, 1, 8>(g, stream) : launch_tile<1, 4, 8>(g, stream);
  if (4 * tiles <= cus) return launch_tile<4, 1, 8>(g, stream);
  return tiles <= cus ? launch_tile<4, 4, 8>(g, stream) : launch_tile<4, 4, 4>(g, stream);
}

}  // namespace mx
