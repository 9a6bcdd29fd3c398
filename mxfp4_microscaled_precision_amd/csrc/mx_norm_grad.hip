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
// rows in a fixed order (no atomics).
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
// norm_grad_wide_kernel.
template <int F32, int V>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormGradArgs a) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  const float inv_n = 1.0f / (float)a.cols;
  float w[V][8], dw[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int64_t c = ((int64_t)u * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[u][i] = dw[u][i] = 0.f;
    if (c < a.cols) load_weight8(a.weight, a.wf32, c, w[u]);
  }
  int flip = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, flip ^= 1) {
    const float rs = a.rstd[r];
    float xh[V][8], dy[V][8];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int64_t c = ((int64_t)u * blockDim.x + threadIdx.x) * 8;
      if (c < a.cols) {
        widen8<F32>(load8<F32>(a.h, r * a.ldh + c), xh[u]);
        widen8<F32>(load8<F32>(a.dy, r * a.lddy + c), dy[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[u][i] *= rs;
          dw[u][i] = __fmaf_rn(dy[u][i], xh[u][i], dw[u][i]);
          dy[u][i] *= w[u][i];
          dot = __fmaf_rn(dy[u][i], xh[u][i], dot);
        }
      }
    }
    const float m = group_sum(dot, part[flip], waves) * inv_n;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int64_t c = ((int64_t)u * blockDim.x + threadIdx.x) * 8;
      if (c < a.cols) {
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (a.dres) widen8<F32>(load8<F32>(a.dres, r * a.ldres + c), o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __fmaf_rn(__fmaf_rn(xh[u][i], -m, dy[u][i]), rs, o[i]);
        store8<F32>(a.dh, r * a.lddh + c, narrow8<F32>(o));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int64_t c = ((int64_t)u * blockDim.x + threadIdx.x) * 8;
    if (c < a.cols) store8<1>(a.partial, (int64_t)blockIdx.x * a.cols + c, narrow8<1>(dw[u]));
  }
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

// dweight[c] = sum of the partial rows, in 64 bits: 64 columns per workgroup,
// four waves share the rows.
__global__ __launch_bounds__(256) void norm_grad_sum_kernel(const float *partial, int groups,
                                                            int64_t cols, float *dweight) {
  __shared__ double part[4][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  double s = 0.0;
  if (c < cols)
    for (int g = wv; g < groups; g += 4) s += (double)partial[(int64_t)g * cols + c];
  part[wv][lane] = s;
  __syncthreads();
  if (wv == 0 && c < cols)
    dweight[c] = (float)((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

template <int F32>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t stream) {
  const int64_t units = (a.cols + 7) / 8;
  const int threads = (int)std::min<int64_t>(1024, (units + 63) / 64 * 64);
  const dim3 grid((unsigned)norm_grad_groups(a.rows));
  hipError_t e = hipSuccess;
  if (a.rows == 0)
    e = hipSuccess;                                    // the sum below writes zeros
  else if (units <= threads)
    e = launch(norm_grad_kernel<F32, 1>, grid, dim3(threads), 0, stream, a);
  else
    e = launch(norm_grad_wide_kernel<F32>, grid, dim3(threads), 0, stream, a);
  if (e != hipSuccess) return e;
  return launch(norm_grad_sum_kernel, dim3((unsigned)((a.cols + 63) / 64)), dim3(256), 0, stream,
                a.partial, (int)grid.x, a.cols, a.dweight);
}

}  // namespace

hipError_t norm_grad_launch(const NormGradArgs &a, hipStream_t stream) {
  return a.f32 ? launch_grad<1>(a, stream) : launch_grad<0>(a, stream);
}

}  // namespace mx
