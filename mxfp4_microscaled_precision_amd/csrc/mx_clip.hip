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
//
// 218 M fp32 elements in nine tensors: 136 us for the squares (872 MB,
// 6.4 TB/s) and 291 us for the scaling (1745 MB, 6.0 TB/s); 111 M bf16
// elements in 288 tensors, none aligned: 41 and 80 us. Bound by HBM and, for
// what is read again, the Infinity cache. (Without vector loads said to be of
// global memory, four of them in flight, and stores past the caches the two
// sets took 517 and 186 us.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

namespace {

constexpr int kThreads = 256;
// Five workgroups to a compute unit (102 registers), which kGradGroups fills on
// 256 of them.
constexpr int kWavesPerSimd = 5;
constexpr int64_t kInfinityCache = (int64_t)256 << 20;

// Tensor addresses come out of a table: said to be global memory, they are
// not looked up as LDS or scratch first.
typedef __attribute__((address_space(1))) uint8_t gbyte;
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef __attribute__((address_space(1))) any_u32x4 g_u32x4;

// Sixteen bytes from any element-aligned address (gfx950 loads and stores them
// at any alignment): 4 fp32 or 8 bf16 elements. Stores, and loads with ONCE, are of data that is not read again here.
template <bool ONCE>
__device__ __forceinline__ any_u32x4 load16(const gbyte *p) {
  const g_u32x4 *q = reinterpret_cast<const g_u32x4 *>(p);
  return ONCE ? __builtin_nontemporal_load(q) : *q;
}
__device__ __forceinline__ void store16(gbyte *p, any_u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<g_u32x4 *>(p));
}

template <int F32>
constexpr int unit_elems() { return F32 ? 4 : 8; }

template <int F32>
__device__ __forceinline__ void widen16(any_u32x4 r, float (&v)[unit_elems<F32>()]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = bits_f(r[i]);
    } else {
      v[2 * i] = bits_f(r[i] << 16);
      v[2 * i + 1] = bits_f(r[i] & 0xFFFF0000u);
    }
  }
}

template <int F32>
__device__ __forceinline__ any_u32x4 narrow16(const float (&v)[unit_elems<F32>()]) {
  any_u32x4 r;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = f_bits(v[i]);
  } else {
    r = narrow8<0>(v).w[0];
  }
  return r;
}

template <int F32>
__device__ __forceinline__ float load_one(const gbyte *p) {
  if (F32) return *reinterpret_cast<const __attribute__((address_space(1))) float *>(p);
  return bits_f((uint32_t)*reinterpret_cast<const __attribute__((address_space(1))) uint16_t *>(p)
                << 16);
}

template <int F32>
__device__ __forceinline__ void store_one(gbyte *p, float v) {
  if constexpr (F32) {
    *reinterpret_cast<__attribute__((address_space(1))) float *>(p) = v;
  } else {
    const float f[8] = {v, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<__attribute__((address_space(1))) uint16_t *>(p) =
        (uint16_t)narrow8<0>(f).w[0][0];
  }
}

// A chunk's elements as contiguous runs: the whole chunk of a tensor without
// gaps, else the piece of each row. f(first element within the tensor's
// buffer, within the tensor, elements, thread, threads); a run of a tensor
// with gaps goes to one wave, a whole chunk to the workgroup. Rows of fewer than
// a wave's units leave lanes idle: norm and scaling of 67 MB in fp32 rows of 256
// take 49 us, but of 33.5 MB in bf16 rows of 64 105 us, of 4 MB in single
// elements 487 us.
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

// A thread's 16-byte units of a run, kBatch of them in flight at a time: f of
// each unit's offset (bytes) and contents; then one element each of the last
// few to g. (Starting the units at the run's first 16-byte boundary instead
// gained nothing on tensors packed without alignment.)
constexpr int kBatch = 4;

template <int F32, bool ONCE, typename F, typename G>
__device__ __forceinline__ void for_units(const gbyte *p, int len, int tid, int threads, F f, G g) {
  constexpr int kSize = F32 ? 4 : 2;
  const int whole = (len * kSize) & ~15, step = threads * 16;
  int i = tid * 16;
  for (; i + (kBatch - 1) * step < whole; i += kBatch * step) {
    any_u32x4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = load16<ONCE>(p + (uint32_t)(i + b * step));
#pragma unroll
    for (int b = 0; b < kBatch; ++b) f(i + b * step, v[b]);
  }
  for (; i < whole; i += step) f(i, load16<ONCE>(p + (uint32_t)i));
  i = whole + tid * kSize;
  if (i < len * kSize) g(i, load_one<F32>(p + (uint32_t)i));
}

template <int F32, bool ONCE>
__device__ __forceinline__ double run_squares(const gbyte *p, int len, int tid, int threads) {
  double acc = 0.0;
  for_units<F32, ONCE>(
      p, len, tid, threads,
      [&](int, any_u32x4 r) {
        float v[unit_elems<F32>()];
        widen16<F32>(r, v);
#pragma unroll
        for (int k = 0; k < unit_elems<F32>(); ++k)
          acc = __builtin_fma((double)v[k], (double)v[k], acc);
      },
      [&](int, float v) { acc = __builtin_fma((double)v, (double)v, acc); });
  return acc;
}

template <int F32, bool ONCE>
__device__ __forceinline__ void run_scale(const gbyte *p, gbyte *o, int len, int tid, int threads,
                                          float coef) {
  for_units<F32, ONCE>(
      p, len, tid, threads,
      [&](int i, any_u32x4 r) {
        float v[unit_elems<F32>()];
        widen16<F32>(r, v);
#pragma unroll
        for (int k = 0; k < unit_elems<F32>(); ++k) v[k] = __fmul_rn(v[k], coef);
        store16(o + (uint32_t)i, narrow16<F32>(v));
      },
      [&](int i, float v) { store_one<F32>(o + (uint32_t)i, __fmul_rn(v, coef)); });
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

// Chunk k of a table: its tensor, its place in it, and how many elements.
struct Chunk {
  GradTensor t;
  uint32_t tensor;
  int64_t first, len;
};

__device__ __forceinline__ Chunk chunk_at(const GradTable &t, int64_t k) {
  const GradChunk c = t.chunk_of[k];
  Chunk r;
  r.t = t.tensors[c.tensor];
  r.tensor = c.tensor;
  r.first = (int64_t)c.at * t.chunk;
  r.len = min(t.chunk, r.t.rows * r.t.cols - r.first);
  return r;
}

__global__ __launch_bounds__(kThreads, kWavesPerSimd) void grad_squares_kernel(GradTable t,
                                                                               double *partial) {
  __shared__ double part[kThreads / 64];
  double acc = 0.0;
  Chunk next = chunk_at(t, blockIdx.x);
  for (int64_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const Chunk c = next;
    next = chunk_at(t, min(k + gridDim.x, t.chunks - 1));   // looked up while this one is read
    const gbyte *base = (const gbyte *)c.t.data;
    for_runs(c.t, c.t.ld, c.first, c.len, [&](int64_t at, int64_t, int64_t n, int tid, int threads) {
      if (k < t.once)
        acc += c.t.f32 ? run_squares<1, true>(base + at * 4, (int)n, tid, threads)
                       : run_squares<0, true>(base + at * 2, (int)n, tid, threads);
      else
        acc += c.t.f32 ? run_squares<1, false>(base + at * 4, (int)n, tid, threads)
                       : run_squares<0, false>(base + at * 2, (int)n, tid, threads);
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
__global__ __launch_bounds__(kThreads, kWavesPerSimd) void grad_scale_kernel(
    GradTable in, GradTable out, const double *partial, int groups, float max_norm, float *norm) {
  __shared__ double part[kThreads / 64];
  const double n = __builtin_sqrt(total_of(partial, groups, part));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // a norm that is NaN makes every element NaN; an infinite one zeroes the
  // finite elements, but not where max_norm is infinite too (no limit)
  const double q = (double)max_norm / (n + 1e-6);
  const bool within = q > 1.0 || (max_norm == __builtin_inff() && n == __builtin_inf());
  const float coef = within ? 1.0f : (float)q;
  if (coef == 1.0f && in.tensors == out.tensors) return;   // nothing changes in place
  const int64_t last = in.chunks - 1;
  Chunk next = chunk_at(in, last - blockIdx.x);           // from the end, see grad_clip_launch
  for (int64_t k = blockIdx.x; k < in.chunks; k += gridDim.x) {
    const Chunk c = next;
    const GradTensor g = c.t, o = out.tensors[c.tensor];
    next = chunk_at(in, last - min(k + gridDim.x, last));
    const gbyte *src = (const gbyte *)g.data;
    gbyte *dst = (gbyte *)o.data;
    // runs without gaps on both sides: the input's, or where that has none the
    // output's
    const int64_t ld = g.ld == g.cols ? o.ld : g.ld;
    for_runs(g, ld, c.first, c.len, [&](int64_t, int64_t e, int64_t m, int tid, int threads) {
      const int64_t r = ld == g.cols ? 0 : e / g.cols, col = e - r * g.cols;
      const int64_t is = ld == g.cols ? e : r * g.ld + col, os = ld == g.cols ? e : r * o.ld + col;
      if (g.f32)
        run_scale<1, true>(src + is * 4, dst + os * 4, (int)m, tid, threads, coef);
      else
        run_scale<0, true>(src + is * 2, dst + os * 2, (int)m, tid, threads, coef);
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

hipError_t grad_clip_launch(const GradTable &all, const GradTable &out, double *partial,
                            float max_norm, float *norm, hipStream_t stream) {
  const int groups = (int)std::min<int64_t>(all.chunks, kGradGroups);
  if (groups == 0) return grad_norm_launch(all, partial, norm, stream);
  // The norm's pass leaves the last 256 MB it reads in the Infinity cache and
  // keeps what comes before out of it; the scaling starts from the end. Read
  // without regard to that a block's gradients took 454 us (fp32) and 211 us
  // (bf16) against 431 us and 208 us, with nothing kept 448 us and 219 us; the
  // small sets that fit as a whole 138 us with nothing kept, 123 us with all.
  GradTable in = all;
  const double kept = (double)kInfinityCache / (double)in.bytes * (double)in.chunks;
  in.once = in.chunks - (kept < (double)in.chunks ? (int64_t)kept : in.chunks);
  const hipError_t e =
      launch(grad_squares_kernel, dim3(groups), dim3(kThreads), 0, stream, in, partial);
  if (e != hipSuccess) return e;
  return launch(grad_scale_kernel, dim3(groups), dim3(kThreads), 0, stream, in, out, partial,
                groups, max_norm, norm);
}

}  // namespace mx
