// What a product's epilogue computes, in fp32 from the accumulator to the one
// rounding of each output:
//
//   forward    z = acc + bias;  pre = z;  C = act(z) * mul + residual
//   gradient   C = acc * mul * act'(pre);  dmul = acc * act(pre)
//
// mul, residual, pre and C are read and written 16 bytes at a time, at any
// alignment: a lane of the tile kernel takes a unit (8 bf16 or 4 fp32 columns of a
// row), one of the few-rows kernel 8 columns of a row. Where the columns of a wave's
// part (of the few-rows kernel's workgroup) are not all the matrix's, or its rows
// are 16 MB or more apart (EpiArgs.vec), a lane takes one column of four rows
// instead, so that the lanes still access adjacent columns. Which activation it is
// is a wave-uniform branch in the few-rows kernel, around all of a lane's elements;
// the tile kernel is compiled for each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

// Direction of an epilogue, constant where the tile kernel's registers depend on
// it: forward with at most one of mul and the residual, or with both; a gradient
// without and with mul.
enum { kForward = 0, kForwardBoth = 1, kGradient = 2, kGradientMul = 3 };
constexpr bool is_gradient(int mode) { return mode >= kGradient; }

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-u): the hardware's exponential and reciprocal (1 ulp each); a
// full-precision division and expf would be some 25 instructions where these
// are four, and a 256x256 tile evaluates 65536 of them.
__device__ __forceinline__ float logistic(float u) {
  return rcp_hw(1.0f + exp2_hw(-kLog2e * u));
}

// e^(-z^2/2) in e and erfc(|z| / sqrt 2) as the result: Abramowitz and Stegun,
// formula 7.1.26 (absolute error at most 1.5e-7, five multiply-adds).
__device__ __forceinline__ float erfc_scaled(float z, float &e) {
  const float x = 0.70710678f * fabsf(z);
  e = exp2_hw(-kLog2e * x * x);
  const float t = rcp_hw(__builtin_fmaf(0.3275911f, x, 1.0f));
  float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  p = __builtin_fmaf(p, t, 1.421413741f);
  p = __builtin_fmaf(p, t, -0.284496736f);
  p = __builtin_fmaf(p, t, 0.254829592f);
  return p * t * e;
}

// tanh form of GELU: z times the logistic function of u = 2 sqrt(2/pi) (z +
// 0.044715 z^3), as (1 + tanh v) / 2 is the logistic function of 2 v.
constexpr float kGelu1 = 1.59576912f, kGelu3 = 0.0713548163f;

// z, but -1e30 for what is below it (NaN stays NaN): the limit of z p at -inf is
// then 0 where the formula has -inf * 0. One v_maximum3_f32.
__device__ __forceinline__ float from_below(float z) {
  return __builtin_elementwise_maximum(z, -1e30f);
}

// act(z). The limits at the infinities; NaN stays NaN.
template <int act>
__device__ __forceinline__ float act_value(float z) {
  if (act == MX_K_ACT_SILU) return from_below(z) * logistic(z);
  if (act == MX_K_ACT_GELU_TANH)
    return from_below(z) * logistic(z * __builtin_fmaf(kGelu3 * z, z, kGelu1));
  if (act == MX_K_ACT_NONE) return z;
  const float up = __builtin_elementwise_maximum(z, 0.0f);
  if (act == MX_K_ACT_RELU) return up;
  // exact GELU: z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2 (no difference
  // of near numbers below zero; from |z| = 64 on the second term is 0)
  float e;
  const float c = erfc_scaled(z, e);
  return __builtin_fmaf(-0.5f * __builtin_amdgcn_fmed3f(fabsf(z), 0.0f, 64.0f), c, up);
}

// act(z) and act'(z). Beyond +-64 the slopes are 0 and 1 in fp32, so the clamp
// only keeps infinity * 0 away (a NaN comes back through p or c).
template <int act>
__device__ __forceinline__ float act_both(float z, float &slope) {
  const float zc = __builtin_amdgcn_fmed3f(z, -64.0f, 64.0f);
  if (act == MX_K_ACT_SILU) {              // slope p + z p (1 - p)
    const float p = logistic(z);
    slope = __builtin_fmaf(zc * p, 1.0f - p, p);
    return from_below(z) * p;
  }
  if (act == MX_K_ACT_GELU_TANH) {         // slope p + z p (1 - p) u'
    const float p = logistic(z * __builtin_fmaf(kGelu3 * z, z, kGelu1));
    const float du = __builtin_fmaf(3.0f * kGelu3 * zc, zc, kGelu1);
    slope = __builtin_fmaf(zc * p * (1.0f - p), du, p);
    return from_below(z) * p;
  }
  slope = 1.0f;
  if (act == MX_K_ACT_NONE) return z;
  const float up = __builtin_elementwise_maximum(z, 0.0f);
  if (act == MX_K_ACT_RELU) {
    slope = z > 0.0f ? 1.0f : up;          // (up: 0, but NaN for NaN)
    return up;
  }
  float e;                                 // slope Phi(z) + z phi(z)
  const float c = 0.5f * erfc_scaled(z, e);
  slope = __builtin_fmaf(zc * 0.398942280f, e, z > 0.0f ? 1.0f - c : c);
  return __builtin_fmaf(-fabsf(zc), c, up);
}

// Calls f with the activation as a constant: one branch where f's elements
// would otherwise branch each (and wait for each other's exponentials).
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case MX_K_ACT_RELU: f(std::integral_constant<int, MX_K_ACT_RELU>()); break;
    case MX_K_ACT_SILU: f(std::integral_constant<int, MX_K_ACT_SILU>()); break;
    case MX_K_ACT_GELU: f(std::integral_constant<int, MX_K_ACT_GELU>()); break;
    case MX_K_ACT_GELU_TANH: f(std::integral_constant<int, MX_K_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, MX_K_ACT_NONE>()); break;
  }
}

// A unit is 16 bytes of a row: 8 bf16 elements or 4 fp32 ones.
template <int F32>
constexpr int kUnit = F32 ? 4 : 8;

template <int F32>
__device__ __forceinline__ float unit_element(const row_u32x4 &r, int i) {
  if constexpr (F32)
    return bits_f(r[i]);
  else
    return bits_f(i & 1 ? r[i >> 1] & 0xFFFF0000u : r[i >> 1] << 16);
}

// Elements i .. i + N - 1, rounded to the unit's type.
template <int F32, int N>
__device__ __forceinline__ void unit_put(row_u32x4 &r, int i, const float (&x)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += F32 ? 1 : 2) {
    if constexpr (F32) {
      r[i + k] = f_bits(x[k]);
    } else {
      typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
      typedef float f2 __attribute__((ext_vector_type(2)));
      r[(i + k) >> 1] =
          __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x[k], x[k + 1]}), bf2));
    }
  }
}

// The epilogue of N elements: v their sums (the bias added), m(k) their mul, o(k)
// their residual (pre, for a gradient); a becomes C, b pre (dmul, for a gradient).
template <int MODE, int ACT, int N, typename M, typename O>
__device__ __forceinline__ void epilogue_of(const float (&v)[N], M m, O o, bool has_mul,
                                            bool has_residual, float (&a)[N], float (&b)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (is_gradient(MODE)) {
      float slope;
      b[k] = v[k] * act_both<ACT>(o(k), slope);
      a[k] = v[k] * slope;
    } else {
      b[k] = v[k];
      a[k] = act_value<ACT>(v[k]);
    }
  }
  if (MODE == kGradientMul || (!is_gradient(MODE) && has_mul)) {
#pragma unroll
    for (int k = 0; k < N; ++k) a[k] *= m(k);
  }
  if (!is_gradient(MODE) && has_residual) {
#pragma unroll
    for (int k = 0; k < N; ++k) a[k] += o(k);
  }
}

// The same of one unit, as stored. Four elements at a time (two of a gradient's):
// enough to overlap their exponentials, and little that is live besides the sums
// (a wave of the tile kernel holds 128 of them).
template <int F32, int MODE, int ACT>
__device__ __forceinline__ void epilogue_unit(const float (&v)[kUnit<F32>], bool has_mul,
                                              bool has_residual, const row_u32x4 &mul,
                                              const row_u32x4 &other, row_u32x4 &c,
                                              row_u32x4 &second) {
  constexpr int n = is_gradient(MODE) ? 2 : 4;
#pragma unroll
  for (int i = 0; i < kUnit<F32>; i += n) {
    float x[n], a[n], b[n];
#pragma unroll
    for (int k = 0; k < n; ++k) x[k] = v[i + k];
    epilogue_of<MODE, ACT>(
        x, [&](int k) { return unit_element<F32>(mul, i + k); },
        [&](int k) { return unit_element<F32>(other, i + k); }, has_mul, has_residual, a, b);
    unit_put<F32>(second, i, b);
    unit_put<F32>(c, i, a);
    if (is_gradient(MODE)) __builtin_amdgcn_sched_barrier(0);
  }
}

// Eight elements as one unit of bf16 or two of fp32.
template <int F32, bool GRAD, int ACT>
__device__ __forceinline__ void epilogue8(const float (&v)[8], const float (&bias)[8], bool has_mul,
                                          bool has_residual, const Row8<F32> &mul,
                                          const Row8<F32> &other, Row8<F32> &c, Row8<F32> &second) {
  constexpr int n = kUnit<F32>;
#pragma unroll
  for (int h = 0; h < 8 / n; ++h) {
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = GRAD ? v[n * h + i] : v[n * h + i] + bias[n * h + i];
    if (GRAD && !has_mul)
      epilogue_unit<F32, kGradient, ACT>(x, false, false, mul.w[h], other.w[h], c.w[h],
                                         second.w[h]);
    else
      epilogue_unit<F32, GRAD ? kGradientMul : kForwardBoth, ACT>(
          x, has_mul, has_residual, mul.w[h], other.w[h], c.w[h], second.w[h]);
  }
}

// The second output, and what `other` is read from.
template <bool GRAD>
__device__ __forceinline__ void *second_of(const EpiArgs &e) {
  return GRAD ? e.dmul : e.pre;
}
template <bool GRAD>
__device__ __forceinline__ int64_t second_ld(const EpiArgs &e) {
  return GRAD ? e.lddmul : e.ldpre;
}
template <bool GRAD>
__device__ __forceinline__ const void *other_of(const EpiArgs &e) {
  return GRAD ? e.pre : e.residual;
}
template <bool GRAD>
__device__ __forceinline__ int64_t other_ld(const EpiArgs &e) {
  return GRAD ? e.ldpre : e.ldres;
}

// Eight consecutive columns of a row, from any element on: gfx950 loads and stores
// 16 bytes at any alignment.
typedef uint32_t any_row_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
template <int F32>
__device__ __forceinline__ Row8<F32> load_row8(const void *p, int64_t at) {
  const any_row_u32x4 *from = reinterpret_cast<const any_row_u32x4 *>(
      static_cast<const uint8_t *>(p) + at * (F32 ? 4 : 2));
  Row8<F32> r;
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) r.w[k] = from[k];
  return r;
}
template <int F32>
__device__ __forceinline__ void store_row8(void *p, int64_t at, const Row8<F32> &r) {
  any_row_u32x4 *to =
      reinterpret_cast<any_row_u32x4 *>(static_cast<uint8_t *>(p) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) to[k] = r.w[k];
}

// One element, widened, and back.
template <int F32>
__device__ __forceinline__ float load_one(const void *p, int64_t at) {
  return F32 ? static_cast<const float *>(p)[at]
             : bits_f((uint32_t) static_cast<const uint16_t *>(p)[at] << 16);
}
template <int F32>
__device__ __forceinline__ void store_one(void *p, int64_t at, float v) {
  if constexpr (F32)
    static_cast<float *>(p)[at] = v;
  else
    static_cast<__bf16 *>(p)[at] = (__bf16)v;
}

// Bias of one column (element `at` of all groups' biases).
__device__ __forceinline__ float load_bias(const EpiArgs &e, int64_t at) {
  return e.bias_f32 ? static_cast<const float *>(e.bias)[at]
                    : bits_f((uint32_t) static_cast<const uint16_t *>(e.bias)[at] << 16);
}

}  // namespace mx
