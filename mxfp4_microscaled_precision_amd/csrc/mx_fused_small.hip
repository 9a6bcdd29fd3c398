// Products with an epilogue and products grouped by expert, where there are
// few rows: MXFP4 operands in the packed tile layout (see mxfp4.h), fp32 sums.
//
// With few rows a product is bound by reading the weights once, and a 256-wide
// tile per compute unit would leave most of the card idle. Here a workgroup
// takes 64 columns of 16 or 64 rows and splits the reduction over its waves:
// wave w reads slices w, w + W, .. straight from memory into registers (a
// tile of the layout is one contiguous 1 KB load of 16 bytes per lane, which
// is the matrix instruction's fragment), and the waves' sums meet in LDS,
// added in wave order, before the epilogue.
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

constexpr int kWaves = 8;
constexpr int kCols = 64;                          // columns of a workgroup's tile
constexpr int kPitch = kCols + 4;                  // LDS row of fp32 sums, 16 bytes of padding

// What a wave reads of one 128-deep slice: R row groups of A, four of B, and
// the scales of the four row groups that each sits among.
template <int R>
struct Slice {
  uint4 a[R], b[4];
  uint32_t sa, sb;
};

template <int R, int F32, bool GRAD>
__global__ __launch_bounds__(64 * kWaves) void fused_small_kernel(FusedArgs g, int row_tiles) {
  constexpr int kRows = 16 * R;
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

  v4f acc[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int ga = ra >> 4, gb = rb >> 4;
  const uint8_t *pa = g.a_codes + ((int64_t)ga * g.a_slices + ka) * 1024 + lane * 16;
  const uint8_t *pb = g.b_codes + ((int64_t)gb * g.b_slices + kb) * 1024 + lane * 16;
  const uint8_t *qa = g.a_scales + ((int64_t)ka * g.a_panels + (ga >> 4)) * 1024 +
                      ((ga >> 2) & 3) * 256 + lane * 4;
  const uint8_t *qb = g.b_scales + ((int64_t)kb * g.b_panels + (gb >> 4)) * 1024 +
                      ((gb >> 2) & 3) * 256 + lane * 4;
  auto read = [&](Slice<R> &s, int k) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s.b[j] = *reinterpret_cast<const uint4 *>(pb + ((int64_t)j * g.b_slices + k) * 1024);
#pragma unroll
    for (int i = 0; i < R; ++i)
      s.a[i] = *reinterpret_cast<const uint4 *>(pa + ((int64_t)i * g.a_slices + k) * 1024);
    s.sb = *reinterpret_cast<const uint32_t *>(qb + (int64_t)k * g.b_panels * 1024);
    s.sa = *reinterpret_cast<const uint32_t *>(qa + (int64_t)k * g.a_panels * 1024);
  };
  auto multiply = [&](const Slice<R> &s) {
    // one row group: its byte of the four comes to the front
    const uint32_t sa = R == 1 ? s.sa >> (8 * (ga & 3)) : s.sa;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // (the byte select is part of the instruction)
#define MX_ROW(I)                                                              \
  if (i == I) {                                                                \
    acc[i][0] = mfma_fp4<0, I>(s.b[0], s.a[i], acc[i][0], s.sb, sa);           \
    acc[i][1] = mfma_fp4<1, I>(s.b[1], s.a[i], acc[i][1], s.sb, sa);           \
    acc[i][2] = mfma_fp4<2, I>(s.b[2], s.a[i], acc[i][2], s.sb, sa);           \
    acc[i][3] = mfma_fp4<3, I>(s.b[3], s.a[i], acc[i][3], s.sb, sa);           \
  }
      MX_ROW(0) MX_ROW(1) MX_ROW(2) MX_ROW(3)
#undef MX_ROW
    }
  };
  // two slices ahead of the one that is multiplied
  Slice<R> s0, s1;
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
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<v4f *>(&red[wave][16 * i + lr][16 * j + 4 * lg]) = acc[i][j];

  // thread -> eight columns of one row
  const int row = ra + (tid >> 3), c8 = (tid & 7) * 8, col = col0 + c8;
  const int lo = max(0, -col), hi = min(8, g.N - col);
  const bool live = tid < kRows * 8 && row >= first && row < last && lo < hi;
  const bool vec = g.e.vec && lo == 0 && hi == 8 && (col & 7) == 0;
  Row8<F32> mul, other, c, second;
  float bias[8];
  if (live) {
    if (g.e.mul) mul = load_cols<F32>(g.e.mul, (c_row + row) * g.e.ldmul + col, vec, lo, hi);
    if (other_of<GRAD>(g.e))
      other = load_cols<F32>(other_of<GRAD>(g.e), (c_row + row) * other_ld<GRAD>(g.e) + col, vec,
                             lo, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      bias[i] = g.e.bias && i >= lo && i < hi ? load_bias(g.e, (int64_t)e * g.N + col + i) : 0.0f;
  }
  __syncthreads();
  if (!live) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float *p = &red[w][tid >> 3][c8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4f d = *reinterpret_cast<const v4f *>(p + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] += d[i];
    }
  }
  with_act(g.e.act, [&](auto act) {
    epilogue8<F32, GRAD, act()>(v, bias, g.e.mul, g.e.residual, mul, other, c, second);
  });
  if (second_of<GRAD>(g.e))
    store_cols<F32>(second_of<GRAD>(g.e), (c_row + row) * second_ld<GRAD>(g.e) + col, vec, lo, hi,
                    second);
  store_cols<F32>(g.c, (c_row + row) * g.ldc + col, vec, lo, hi, c);
}

template <int R, int F32, bool GRAD>
hipError_t launch_small(const FusedArgs &g, hipStream_t stream) {
  constexpr int kRows = 16 * R;
  const int64_t tm = ((int64_t)g.M + kRows - 1) / kRows;
  // a group's tiles begin at a multiple of kRows: up to two more than its rows'
  int64_t rt = tm;
  if (g.kind == MX_K_WGRAD)
    rt = tm * g.groups;
  else if (g.ends)
    rt = g.rows / kRows + 2 * (int64_t)std::min(g.groups, g.rows);
  int64_t ct = ((int64_t)g.N + kCols - 1) / kCols;
  if (g.kind == MX_K_FPROP && g.groups > 1 && g.N % kCols) ++ct;   // unaligned first columns
  if (rt * ct == 0) return hipSuccess;
  if (rt * ct > INT32_MAX) return hipErrorInvalidValue;
  return launch(fused_small_kernel<R, F32, GRAD>, dim3((unsigned)(rt * ct)), dim3(64 * kWaves), 0,
                stream, g, (int)rt);
}

template <int R>
hipError_t launch_rows(const FusedArgs &g, hipStream_t stream) {
  if (g.grad)
    return g.out_bf16 ? launch_small<R, 0, true>(g, stream) : launch_small<R, 1, true>(g, stream);
  return g.out_bf16 ? launch_small<R, 0, false>(g, stream) : launch_small<R, 1, false>(g, stream);
}

}  // namespace

hipError_t fused_small_launch(const FusedArgs &g, hipStream_t stream) {
  return g.M <= 16 ? launch_rows<1>(g, stream) : launch_rows<4>(g, stream);
}

}  // namespace mx
