// The 2-norm over many gradient tensors, and the tensors scaled so that it
// does not exceed max_norm:
//
//   norm = sqrt(sum g^2);   out = g * min(1, max_norm / (norm + 1e-6))
//
// Squares and sums are held in 64 bits: a square of fp32's or bf16's smallest
// or largest value neither vanishes nor overflows there, and the two
// instructions an element costs stay far below what its bytes cost.
//
// The tensors' elements are cut into chunks of one size; a table made once on
// the host says which tensor a chunk lies in. Workgroups walk the chunks with
// the grid's stride and leave one partial sum each; whoever needs the norm
// adds the partial sums in a fixed order (no atomics).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

namespace {

constexpr int kThreads = 256;

// Elements [0, n) of a contiguous run: f(index) for the lanes of a workgroup
// in units of eight, then the last few one by one.
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements from any element-aligned address (gfx950 loads and stores 16
// bytes at any alignment).
template <int F32>
__device__ __forceinline__ Row8<F32> load_any8(const uint8_t *p) {
  Row8<F32> r;
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) r.w[k] = reinterpret_cast<const any_u32x4 *>(p)[k];
  return r;
}

template <int F32>
__device__ __forceinline__ void store_any8(uint8_t *p, const Row8<F32> &r) {
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) reinterpret_cast<any_u32x4 *>(p)[k] = r.w[k];
}

template <int F32>
__device__ __forceinline__ float load_one(const uint8_t *p) {
  if (F32) return *reinterpret_cast<const float *>(p);
  return bits_f((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}

template <int F32>
__device__ __forceinline__ void store_one(uint8_t *p, float v) {
  if constexpr (F32) {
    *reinterpret_cast<float *>(p) = v;
  } else {
    const float f[8] = {v, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<uint16_t *>(p) = (uint16_t)narrow8<0>(f).w[0][0];
  }
}

// A chunk's elements as contiguous runs: the whole chunk of a tensor without
// gaps, else the piece of each row. f(first element within the tensor's
// buffer, elements, thread, threads); a run of a tensor with gaps goes to one
// wave, a whole chunk to the workgroup.
template <typename F>
__device__ __forceinline__ void for_runs(const GradTensor &t, int64_t ld, int64_t first,
                                         int64_t len, F f) {
  if (ld == t.cols) {
    f(first, first, len, (int)threadIdx.x, kThreads);
    return;
  }
  const int64_t r0 = first / t.cols, r1 = (first + len - 1) / t.cols;
  for (int64_t r = r0 + (threadIdx.x >> 6); r <= r1; r += kThreads / 64) {
    const int64_t c0 = r == r0 ? first - r0 * t.cols : 0;
    const int64_t c1 = r == r1 ? first + len - r1 * t.cols : t.cols;
    f(r * ld + c0, r * t.cols + c0, c1 - c0, (int)(threadIdx.x & 63), 64);
  }
}

template <int F32>
__device__ __forceinline__ double run_squares(const uint8_t *p, int64_t len, int tid, int threads) {
  constexpr int kSize = F32 ? 4 : 2;
  double acc = 0.0;
  const int64_t whole = len & ~(int64_t)7;
  for (int64_t i = tid * 8; i < whole; i += threads * 8) {
    float v[8];
    widen8<F32>(load_any8<F32>(p + i * kSize), v);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc = __builtin_fma((double)v[k], (double)v[k], acc);
  }
  if (tid < len - whole) {
    const double v = (double)load_one<F32>(p + (whole + tid) * kSize);
    acc = __builtin_fma(v, v, acc);
  }
  return acc;
}

template <int F32>
__device__ __forceinline__ void run_scale(const uint8_t *p, uint8_t *o, int64_t len, int tid,
                                          int threads, float coef) {
  constexpr int kSize = F32 ? 4 : 2;
  const int64_t whole = len & ~(int64_t)7;
  for (int64_t i = tid * 8; i < whole; i += threads * 8) {
    float v[8];
    widen8<F32>(load_any8<F32>(p + i * kSize), v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], coef);
    store_any8<F32>(o + i * kSize, narrow8<F32>(v));
  }
  if (tid < len - whole)
    store_one<F32>(o + (whole + tid) * kSize,
                   __fmul_rn(load_one<F32>(p + (whole + tid) * kSize), coef));
}

__device__ __forceinline__ double group_sum(double v, double *part) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += part[i];
  return s;
}

// The sum of the partial sums, the same in every workgroup that asks.
__device__ __forceinline__ double total_of(const double *partial, int groups, double *part) {
  double s = 0.0;
  for (int i = threadIdx.x; i < groups; i += kThreads) s += partial[i];
  return group_sum(s, part);
}

__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradTable t, double *partial) {
  __shared__ double part[kThreads / 64];
  double acc = 0.0;
  for (int64_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const GradChunk c = t.chunk_of[k];
    const GradTensor g = t.tensors[c.tensor];
    const int64_t first = (int64_t)c.at * t.chunk, len = min(t.chunk, g.rows * g.cols - first);
    const uint8_t *base = static_cast<const uint8_t *>(g.data);
    for_runs(g, g.ld, first, len, [&](int64_t at, int64_t, int64_t n, int tid, int threads) {
      acc += g.f32 ? run_squares<1>(base + at * 4, n, tid, threads)
                   : run_squares<0>(base + at * 2, n, tid, threads);
    });
  }
  const double s = group_sum(acc, part);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double *partial, int groups,
                                                             float *norm) {
  __shared__ double part[kThreads / 64];
  const double s = total_of(partial, groups, part);
  if (threadIdx.x == 0) *norm = (float)__builtin_sqrt(s);
}

// in and out describe the same shapes and types; they may be the same table.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradTable in, GradTable out,
                                                              const double *partial, int groups,
                                                              float max_norm, float *norm) {
  __shared__ double part[kThreads / 64];
  const double n = __builtin_sqrt(total_of(partial, groups, part));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // a norm that is NaN makes every element NaN; an infinite one zeroes the
  // finite elements
  const double q = (double)max_norm / (n + 1e-6);
  const float coef = q > 1.0 ? 1.0f : (float)q;
  if (coef == 1.0f && in.tensors == out.tensors) return;   // nothing changes in place
  for (int64_t k = blockIdx.x; k < in.chunks; k += gridDim.x) {
    const GradChunk c = in.chunk_of[k];
    const GradTensor g = in.tensors[c.tensor], o = out.tensors[c.tensor];
    const int64_t first = (int64_t)c.at * in.chunk, len = min(in.chunk, g.rows * g.cols - first);
    const uint8_t *src = static_cast<const uint8_t *>(g.data);
    uint8_t *dst = static_cast<uint8_t *>(o.data);
    // runs without gaps on both sides: the input's, or where that has none the
    // output's
    const int64_t ld = g.ld == g.cols ? o.ld : g.ld;
    for_runs(g, ld, first, len, [&](int64_t, int64_t e, int64_t m, int tid, int threads) {
      const int64_t r = ld == g.cols ? 0 : e / g.cols, col = e - r * g.cols;
      const int64_t is = ld == g.cols ? e : r * g.ld + col, os = ld == g.cols ? e : r * o.ld + col;
      if (g.f32)
        run_scale<1>(src + is * 4, dst + os * 4, m, tid, threads, coef);
      else
        run_scale<0>(src + is * 2, dst + os * 2, m, tid, threads, coef);
    });
  }
}

}  // namespace

hipError_t grad_norm_launch(const GradTable &t, double *partial, float *norm, hipStream_t stream) {
  const int groups = (int)std::min<int64_t>(t.chunks, kGradGroups);
  if (groups > 0) {
    const hipError_t e =
        launch(grad_squares_kernel, dim3(groups), dim3(kThreads), 0, stream, t, partial);
    if (e != hipSuccess) return e;
  }
  return launch(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, partial, groups, norm);
}

hipError_t grad_clip_launch(const GradTable &in, const GradTable &out, double *partial,
                            float max_norm, float *norm, hipStream_t stream) {
  const int groups = (int)std::min<int64_t>(in.chunks, kGradGroups);
  if (groups == 0) return grad_norm_launch(in, partial, norm, stream);
  const hipError_t e =
      launch(grad_squares_kernel, dim3(groups), dim3(kThreads), 0, stream, in, partial);
  if (e != hipSuccess) return e;
  return launch(grad_scale_kernel, dim3(groups), dim3(kThreads), 0, stream, in, out, partial,
                groups, max_norm, norm);
}

}  // namespace mx
