// What a product's epilogue computes, eight consecutive columns of one row at
// a time, in fp32 from the accumulator to the one rounding of each output:
//
//   forward    z = acc + bias;  pre = z;  C = act(z) * mul + residual
//   gradient   C = acc * mul * act'(pre);  dmul = acc * act(pre)
//
// A lane owns 8 columns (16 bytes of a bf16 row, 32 of an fp32 one), so mul,
// residual, pre and C are read and written as whole 128-byte row pieces by
// eight lanes; which activation it is is a wave-uniform branch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

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

// act(z). The limits at the infinities; NaN stays NaN. (A product with -1e30
// in -inf's place keeps the limit 0 where the formula has -inf * 0.)
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == MX_K_ACT_SILU) return fmaxf(z, -1e30f) * logistic(z);
  if (act == MX_K_ACT_GELU_TANH)
    return fmaxf(z, -1e30f) * logistic(z * __builtin_fmaf(kGelu3 * z, z, kGelu1));
  if (act == MX_K_ACT_NONE) return z;
  const float up = __builtin_elementwise_maximum(z, 0.0f);
  if (act == MX_K_ACT_RELU) return up;
  // exact GELU: z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2 (no difference
  // of near numbers below zero)
  float e;
  const float c = erfc_scaled(z, e);
  return __builtin_fmaf(-0.5f * fminf(fabsf(z), 64.0f), c, up);
}

// act(z) and act'(z). Beyond +-64 the slopes are 0 and 1 in fp32, so the
// clamp only keeps infinity * 0 away.
__device__ __forceinline__ float act_both(float z, int act, float &slope) {
  const float zc = __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f);
  if (act == MX_K_ACT_SILU || act == MX_K_ACT_GELU_TANH) {
    const bool tanh_form = act == MX_K_ACT_GELU_TANH;
    const float z2 = kGelu3 * zc * zc;
    const float p = logistic(tanh_form ? z * __builtin_fmaf(kGelu3 * z, z, kGelu1) : z);
    const float du = tanh_form ? __builtin_fmaf(3.0f, z2, kGelu1) : 1.0f;
    slope = __builtin_fmaf(zc * p * (1.0f - p), du, p);
    return fmaxf(z, -1e30f) * p;
  }
  slope = 1.0f;
  if (act == MX_K_ACT_NONE) return z;
  const float up = __builtin_elementwise_maximum(z, 0.0f);
  if (act == MX_K_ACT_RELU) {
    slope = z > 0.0f ? 1.0f : 0.0f;
    return up;
  }
  float e;
  const float c = 0.5f * erfc_scaled(z, e);
  slope = __builtin_fmaf(zc * 0.398942280f, e, z > 0.0f ? 1.0f - c : c);
  if (z != z) slope = z;
  return __builtin_fmaf(-fminf(fabsf(z), 64.0f), c, up);
}

// Eight elements of a [.., ld] matrix as stored (F32: fp32, else bf16).
template <int F32>
__device__ __forceinline__ Row8<F32> epi_load(const void *p, int64_t at, bool vec, int lo, int hi) {
  if (vec) return load8<F32>(p, at);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (i >= lo && i < hi)
      v[i] = F32 ? static_cast<const float *>(p)[at + i]
                 : bits_f((uint32_t) static_cast<const uint16_t *>(p)[at + i] << 16);
  }
  return narrow8<F32>(v);
}

template <int F32>
__device__ __forceinline__ void epi_store(void *p, int64_t at, bool vec, int lo, int hi,
                                          const float (&v)[8]) {
  const Row8<F32> r = narrow8<F32>(v);
  if (vec) {
    store8<F32>(p, at, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i >= lo && i < hi) {
      if (F32)
        static_cast<uint32_t *>(p)[at + i] = r.w[i >> 2][i & 3];
      else
        static_cast<uint16_t *>(p)[at + i] = (uint16_t)(r.w[0][i >> 1] >> (16 * (i & 1)));
    }
}

// What the epilogue reads for 8 columns of a row, loaded ahead of its use.
// Columns [lo, hi) of the eight are the output's; `vec`: all of them, at an
// address for 16-byte accesses in every matrix the call has.
template <int F32, bool GRAD>
struct EpiIn {
  Row8<F32> mul, other;          // other: the residual, or pre for a gradient

  __device__ __forceinline__ void load(const EpiArgs &e, int64_t row, int64_t col, bool vec, int lo,
                                       int hi) {
    if (e.mul) mul = epi_load<F32>(e.mul, row * e.ldmul + col, vec, lo, hi);
    if (GRAD)
      other = epi_load<F32>(e.pre, row * e.ldpre + col, vec, lo, hi);
    else if (e.residual)
      other = epi_load<F32>(e.residual, row * e.ldres + col, vec, lo, hi);
  }
};

// Columns [lo, hi) of the 8 from (row, col) on, given their sums v.
template <int F32, bool GRAD>
__device__ __forceinline__ void epilogue8(const EpiArgs &e, void *c, int64_t ldc, float (&v)[8],
                                          const EpiIn<F32, GRAD> &in, const float (&bias)[8],
                                          int64_t row, int64_t col, bool vec, int lo, int hi) {
  float m[8], o[8];
  if (e.mul) widen8<F32>(in.mul, m);
  if (GRAD) {
    widen8<F32>(in.other, o);
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float slope;
      const float y = act_both(o[i], e.act, slope);
      d[i] = v[i] * y;
      v[i] *= slope;
      if (e.mul) v[i] *= m[i];
    }
    if (e.dmul) epi_store<F32>(e.dmul, row * e.lddmul + col, vec, lo, hi, d);
  } else {
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += bias[i];
    }
    if (e.pre) epi_store<F32>(e.pre, row * e.ldpre + col, vec, lo, hi, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], e.act);
    if (e.mul) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= m[i];
    }
    if (e.residual) {
      widen8<F32>(in.other, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += o[i];
    }
  }
  epi_store<F32>(c, row * ldc + col, vec, lo, hi, v);
}

// Bias of 8 columns (of a group's row of biases from element `at` on).
__device__ __forceinline__ void epi_bias(const EpiArgs &e, int64_t at, int lo, int hi,
                                         float (&bias)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = 0.0f;
    if (e.bias && i >= lo && i < hi)
      bias[i] = e.bias_f32 ? static_cast<const float *>(e.bias)[at + i]
                           : bits_f((uint32_t) static_cast<const uint16_t *>(e.bias)[at + i] << 16);
  }
}

}  // namespace mx
