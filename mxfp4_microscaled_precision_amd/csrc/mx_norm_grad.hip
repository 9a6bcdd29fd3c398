// Gradient of the RMS norm for gfx950. With x^ = h * rstd, y = x^ * weight and
// n = cols:
//
//   dh      = rstd * (dy * weight - x^ * mean_k(dy * weight * x^)) + dres
//   dweight = sum over rows of dy * x^
//
// dh is the gradient of the residual stream (and of both terms of its sum);
// dres is what reaches it past the norm. The quantization of y passes its
// gradient through unchanged.
//
// A workgroup walks rows with a stride of the grid: a thread owns the same
// columns of each, so the weight's gradient stays in its registers and one
// partial row per workgroup reaches memory. A second launch adds the partial
// rows in a fixed order (no atomics). A few rows take one launch. Row sums and
// the partial rows are fp32, the sum over workgroups is fp64.
//
// 16384 x 4096 bf16 with dres: 85.4 us for 547 MB (6.4 TB/s: bound by HBM)
// and 4.8 us for the second launch (8 MB of partial rows); before the next
// row's loads overlapped the row sum the two took 106 and 32 us. Wider rows are
// further from their bytes at a copy's 5.4 TB/s: 2048 x 8192 29.8 us against
// 24.9, 2048 x 12288 52.6 against 37.3 (one workgroup of sixteen waves to a
// compute unit), fp32 117.7 against 74.6 and 1024 x 28672 96.3 against 43.5
// (norm_grad_wide_kernel).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

namespace {

// Sum over the workgroup, the same value in every thread. `part` holds one
// float per wave; two of them alternate between calls, so one barrier does.
__device__ __forceinline__ float group_sum(float v, float *part, int waves) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = part[0];
  for (int i = 1; i < waves; ++i) s += part[i];
  return s;
}

// V units of eight columns per thread cover a row in one go; wider rows take
// norm_grad_wide_kernel. The next row's loads are in flight while the
// workgroup adds up this one's products. ONCE: they are kept out of the
// caches.
template <int F32, int V, bool ONCE>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormGradArgs a) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  const float inv_n = 1.0f / (float)a.cols;
  // A unit's 8 columns: adjacent ones (bf16) or two times 4, blockDim.x * 4
  // apart (fp32), so that each access of a wave covers whole lines (8192 x 4096
  // fp32 with dres: 90.9 us, by 8 adjacent columns 105.4 us).
  constexpr int kParts = F32 ? 2 : 1, kPartCols = 8 / kParts;
  float w[V][8], dw[V][8];
  int64_t col[V][kParts];
  bool live[V][kParts];
#pragma unroll
  for (int u = 0; u < V; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[u][i] = dw[u][i] = 0.f;
#pragma unroll
    for (int n = 0; n < kParts; ++n) {
      const int64_t c = ((int64_t)(u * kParts + n) * blockDim.x + threadIdx.x) * kPartCols;
      live[u][n] = c < a.cols;
      // threads past the row read its end and count nothing
      col[u][n] = min(c, a.cols - kPartCols);
      if (!live[u][n]) continue;
      if constexpr (F32)
        load_weight4(a.weight, a.wf32, c, w[u] + 4 * n);
      else
        load_weight8(a.weight, a.wf32, c, w[u]);
    }
  }
  auto load = [&](const void *p, int64_t row0, int u) {
    Row8<F32> v;
#pragma unroll
    for (int n = 0; n < kParts; ++n) v.w[n] = load16<F32, ONCE>(p, row0 + col[u][n]);
    return v;
  };
  Row8<F32> h[V], dy[V], res[V];
  float rs;
  auto read = [&](int64_t r) {
    rs = a.rstd[r];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      h[u] = load(a.h, r * a.ldh, u);
      dy[u] = load(a.dy, r * a.lddy, u);
      if (a.dres) res[u] = load(a.dres, r * a.ldres, u);
    }
  };
  int flip = 0;
  int64_t r = blockIdx.x;
  read(r);
  for (; r < a.rows; r += gridDim.x, flip ^= 1) {
    float xh[V][8], g[V][8];
    Row8<F32> o[V];
    float dot = 0.f;
    const float s = rs;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      widen8<F32>(h[u], xh[u]);
      widen8<F32>(dy[u], g[u]);
      o[u] = res[u];
      float d[kParts] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[u][i] *= s;
        dw[u][i] = __fmaf_rn(g[u][i], xh[u][i], dw[u][i]);
        g[u][i] *= w[u][i];
        d[i / kPartCols] = __fmaf_rn(g[u][i], xh[u][i], d[i / kPartCols]);
      }
#pragma unroll
      for (int n = 0; n < kParts; ++n) dot += live[u][n] ? d[n] : 0.f;
    }
    read(min(r + gridDim.x, a.rows - 1));
    const float m = group_sum(dot, part[flip], waves) * inv_n;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (live[u][0]) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (a.dres) widen8<F32>(o[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fmaf_rn(__fmaf_rn(xh[u][i], -m, g[u][i]), s, f[i]);
        const Row8<F32> v = narrow8<F32>(f);
#pragma unroll
        for (int n = 0; n < kParts; ++n)
          if (live[u][n]) store16<F32, false>(a.dh, r * a.lddh + col[u][n], v.w[n]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < V; ++u)
#pragma unroll
    for (int n = 0; n < kParts; ++n)
      if (live[u][n])
#pragma unroll
        for (int i = 0; i < kPartCols; i += 4)
          *reinterpret_cast<float4 *>(a.partial + (int64_t)blockIdx.x * a.cols + col[u][n] + i) =
              make_float4(dw[u][n * kPartCols + i], dw[u][n * kPartCols + i + 1],
                          dw[u][n * kPartCols + i + 2], dw[u][n * kPartCols + i + 3]);
}

// Rows of any width: two passes over the row, the second from cache, and the
// partial weight gradient kept in memory. Each thread reads back only what it
// has written itself.
template <int F32>
__global__ __launch_bounds__(1024) void norm_grad_wide_kernel(NormGradArgs a) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  const float inv_n = 1.0f / (float)a.cols;
  const int64_t p0 = (int64_t)blockIdx.x * a.cols;
  int flip = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, flip ^= 1) {
    const float rs = a.rstd[r];
    const bool first = r == blockIdx.x;
    float dot = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += blockDim.x * 8) {
      float x[8], d[8], w[8], p[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      widen8<F32>(load8<F32>(a.h, r * a.ldh + c), x);
      widen8<F32>(load8<F32>(a.dy, r * a.lddy + c), d);
      load_weight8(a.weight, a.wf32, c, w);
      if (!first) widen8<1>(load8<1>(a.partial, p0 + c), p);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= rs;
        p[i] = __fmaf_rn(d[i], x[i], p[i]);
        dot = __fmaf_rn(d[i] * w[i], x[i], dot);
      }
      store8<1>(a.partial, p0 + c, narrow8<1>(p));
    }
    const float m = group_sum(dot, part[flip], waves) * inv_n;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += blockDim.x * 8) {
      float x[8], d[8], w[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      widen8<F32>(load8<F32>(a.h, r * a.ldh + c), x);
      widen8<F32>(load8<F32>(a.dy, r * a.lddy + c), d);
      load_weight8(a.weight, a.wf32, c, w);
      if (a.dres) widen8<F32>(load8<F32>(a.dres, r * a.ldres + c), o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = __fmaf_rn(__fmaf_rn(x[i] * rs, -m, d[i] * w[i]), rs, o[i]);
      store8<F32>(a.dh, r * a.lddh + c, narrow8<F32>(o));
    }
  }
}

// Few rows in one launch: a workgroup of sixteen waves owns 512 columns. Each
// works out the dot products of all rows by itself (wave w those of rows w and
// w + 16), then dh of its columns, and adds the waves' parts of the weight's
// gradient in LDS.

template <int F32>
__global__ __launch_bounds__(1024) void norm_grad_few_kernel(NormGradArgs a) {
  __shared__ float dots[kFewRows];
  __shared__ __attribute__((aligned(16))) float sums[16][512];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float inv_n = 1.0f / (float)a.cols;
  for (int r = wv; r < a.rows; r += 16) {
    const float rs = a.rstd[r];
    float dot = 0.f;
    for (int64_t c = lane * 8; c < a.cols; c += 512) {
      float x[8], g[8], w[8];
      widen8<F32>(load8<F32>(a.h, r * a.ldh + c), x);
      widen8<F32>(load8<F32>(a.dy, r * a.lddy + c), g);
      load_weight8(a.weight, a.wf32, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = __fmaf_rn(g[i] * w[i], x[i] * rs, dot);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) dot += __shfl_xor(dot, m);
    if (lane == 0) dots[r] = dot * inv_n;
  }
  __syncthreads();
  for (int64_t c0 = (int64_t)blockIdx.x * 512; c0 < a.cols; c0 += (int64_t)gridDim.x * 512) {
    const int64_t c = c0 + lane * 8;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < a.cols) {
      float w[8];
      load_weight8(a.weight, a.wf32, c, w);
      for (int r = wv; r < a.rows; r += 16) {
        const float rs = a.rstd[r], m = dots[r];
        float x[8], g[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        widen8<F32>(load8<F32>(a.h, r * a.ldh + c), x);
        widen8<F32>(load8<F32>(a.dy, r * a.lddy + c), g);
        if (a.dres) widen8<F32>(load8<F32>(a.dres, r * a.ldres + c), o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= rs;
          dw[i] = __fmaf_rn(g[i], x[i], dw[i]);
          o[i] = __fmaf_rn(__fmaf_rn(x[i], -m, g[i] * w[i]), rs, o[i]);
        }
        store8<F32>(a.dh, r * a.lddh + c, narrow8<F32>(o));
      }
    }
    store8<1>(sums[wv], lane * 8, narrow8<1>(dw));
    __syncthreads();
    if (threadIdx.x < 512 && c0 + threadIdx.x < a.cols) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s += sums[i][threadIdx.x];
      a.dweight[c0 + threadIdx.x] = s;
    }
    __syncthreads();                                    // sums is read
  }
}

// dweight[c] = sum of the partial rows (cols apart), c < width, in 64 bits: 32
// columns per workgroup, 32 threads to a column, all of a thread's loads in
// flight together.
__global__ __launch_bounds__(1024) void norm_grad_sum_kernel(const float *partial, int groups,
                                                             int64_t cols, int64_t width,
                                                             float *dweight) {
  __shared__ double part[32][33];
  const int c = threadIdx.x & 31, t = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  double s = 0.0;
  if (col < width) {
    const float *p = partial + col;
    int g = t;
    for (; g + 7 * 32 < groups; g += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[(int64_t)(g + i * 32) * cols];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += (double)v[i];
    }
    for (; g < groups; g += 32) s += (double)p[(int64_t)g * cols];
  }
  part[t][c] = s;
  __syncthreads();
  // thread (t, c) takes row c of column t: half a wave adds a column up
  double v = part[c][t];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) v += __shfl_xor(v, m);
  if (c == 0 && (int64_t)blockIdx.x * 32 + t < width) dweight[(int64_t)blockIdx.x * 32 + t] = (float)v;
}

// One unit of eight columns per thread up to 8192 columns, two of bf16 rows up
// to 16384 (2048 x 12288: 53 us, in two passes 81 us); fp32 rows would spill
// there (198 us against 120 us) and take the two passes.
// Rows that fill three quarters of the 256 MB Infinity cache are read past it
// (16384 x 4096 bf16: 92 us, else 105 us; 2048 x 12288: 53 us, else 56 us);
// smaller ones may be in it from what wrote them (4096 x 1024: 14.0 us, past
// it 15.1 us).
template <int F32, bool ONCE>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t stream) {
  if (norm_grad_few(a.rows, a.cols)) {
    // every workgroup reads all of dy: where dh is written over it, one does
    // all the columns, after its own reads
    const unsigned groups = a.dh == a.dy ? 1u : (unsigned)((a.cols + 511) / 512);
    return launch(norm_grad_few_kernel<F32>, dim3(groups), dim3(1024), 0, stream, a);
  }
  const int64_t units = a.cols / 8;
  const int threads = (int)std::min<int64_t>(1024, (units + 63) / 64 * 64);
  const dim3 grid((unsigned)norm_grad_groups(a.rows, a.cols));
  hipError_t e = hipSuccess;                           // without rows the sum writes zeros
  if (a.rows > 0) {
    if (units <= threads)
      e = launch(norm_grad_kernel<F32, 1, ONCE>, grid, dim3(threads), 0, stream, a);
    else if (!F32 && units <= 2 * threads)
      e = launch(norm_grad_kernel<0, 2, ONCE>, grid, dim3(threads), 0, stream, a);
    else
      e = launch(norm_grad_wide_kernel<F32>, grid, dim3(threads), 0, stream, a);
  }
  // a launch holds fewer than 2^32 threads: 2^26 columns take half of that
  constexpr int64_t kSumCols = (int64_t)1 << 26;
  for (int64_t c = 0; c < a.cols && e == hipSuccess; c += kSumCols) {
    const int64_t width = std::min(kSumCols, a.cols - c);
    e = launch(norm_grad_sum_kernel, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, stream,
               a.partial + c, (int)grid.x, a.cols, width, a.dweight + c);
  }
  return e;
}

}  // namespace

hipError_t norm_grad_launch(const NormGradArgs &a, hipStream_t stream) {
  const bool once =
      a.rows * a.cols * (a.f32 ? 4 : 2) * (a.dres != nullptr ? 4 : 3) >= (int64_t)192 << 20;
  if (a.f32) return once ? launch_grad<1, true>(a, stream) : launch_grad<1, false>(a, stream);
  return once ? launch_grad<0, true>(a, stream) : launch_grad<0, false>(a, stream);
}

}  // namespace mx
