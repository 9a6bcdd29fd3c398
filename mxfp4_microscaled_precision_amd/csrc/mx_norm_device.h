// Pieces shared by the norm's kernels: the residual stream's sum, rstd, the
// weights, and the encoding of one block of y for either operand.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "mx_encode.h"
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

// The row's h from x and the residual: bf16 rows round the sum to bf16 (exact
// in fp32 wherever that matters: fp32 holds two bf16 values less than 16
// binades apart, and beyond that the smaller one is below half a step).
template <int F32>
__device__ __forceinline__ Row8<F32> add_rows(const Row8<F32> &x, const Row8<F32> &r) {
  float a[8], b[8];
  widen8<F32>(x, a);
  widen8<F32>(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = __fadd_rn(a[i], b[i]);
  return narrow8<F32>(a);
}

// acc + v . v in 64 bits, element by element.
__device__ __forceinline__ double add_squares(double acc, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = __builtin_fma((double)v[i], (double)v[i], acc);
  return acc;
}

// 1 / sqrt(sum / n + eps) from the hardware's reciprocal root (some 26 bits)
// and two Newton steps, which take it to about 2^-51: a division and a root of
// full precision would be four times as many dependent instructions, on the
// path of every workgroup. Zero, infinity and NaN are the hardware's result.
__device__ __forceinline__ float rstd_of(double sum, double inv_n, double eps) {
  const double t = __builtin_fma(sum, inv_n, eps);
  double y = __builtin_amdgcn_rsq(t);
  const double half = -0.5 * t;
  if (t > 0.0 && t < __builtin_inf()) {
#pragma unroll
    for (int i = 0; i < 2; ++i) y = __builtin_fma(__builtin_fma(half * y, y, 0.5), y, y);
  }
  return (float)y;
}

// Weights as they lie in memory, loaded ahead of their use.
__device__ __forceinline__ Row8<1> load_weight_raw(const void *w, int f32, int64_t i) {
  if (f32) return load8<1>(w, i);
  Row8<1> r;
  r.w[0] = load8<0>(w, i).w[0];
  r.w[1] = r.w[0];
  return r;
}

__device__ __forceinline__ void widen_weight(const Row8<1> &r, int f32, float (&v)[8]) {
  if (f32) {
    widen8<1>(r, v);
  } else {
    Row8<0> b;
    b.w[0] = r.w[0];
    widen8<0>(b, v);
  }
}

// The block of y of row r at K = 32 kb of the axis-1 operand, rotated (random
// signs: mask) and rounded; returns its scale code. The stochastic rounding
// index is L = r * cols + 32 kb + i (cols % 32 == 0). quantize_block multiplies
// once by c * 2^-e where the rule multiplies twice (nearest rounding): for y of
// more bits than bf16 the two agree unless the value times c is subnormal in
// fp32 (below 2^-126), where they may come out on different sides of a rounding
// border. Such a value has a code other than 0 only in a block whose scale is
// below 2^-115, its largest value below 2^-106 (E4M3; 2^-121 for E2M1).
template <int ROT, int RND, int FMT, int kWords>
__device__ __forceinline__ uint32_t encode_row_block(const NormArgs &a, float (&y)[32], int64_t r,
                                                     int64_t kb, uint32_t mask,
                                                     uint32_t (&out)[kWords]) {
  if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
  rotate_block<ROT>(y);
  const uint64_t q0 = (uint64_t)(r * a.cols + (kb << 5)) >> 2;
  U4 w{0u, 0u, 0u, 0u};
  auto u24_of = [&](int i) -> uint32_t {
    if ((i & 3) == 0) w = sr_words(q0 + (uint64_t)(i >> 2), a.seed1_lo, a.seed1_hi);
    return pick_word(w, (uint32_t)(i & 3)) >> 8;
  };
  return quantize_block<RotKind<ROT>::value, RND, FMT>(y, out, u24_of);
}

// The block of y of column c at rows R0 .. R0 + 31 of the axis-0 operand, as
// above. With stochastic rounding the four lanes of a quad must hold four
// columns c % 4 == 0 .. 3: element (R0 + i, c) draws word c % 4 of the call at
// ((R0 + i) cols + c - c % 4) / 4, so each lane makes the calls of every fourth
// row and a 4 x 4 transpose hands each its column's words.
template <int ROT, int RND, int FMT, int kWords>
__device__ __forceinline__ uint32_t encode_col_block(const NormArgs &a, float (&y)[32], int64_t R0,
                                                     int64_t c, uint32_t mask,
                                                     uint32_t (&out)[kWords]) {
  if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
  rotate_block<ROT>(y);
  if constexpr (RND == MX_K_ROUND_SR) {
    float m1, m2;
    const uint32_t s = block_scale<RotKind<ROT>::value>(y, m1, m2);
    const uint32_t q = (uint32_t)(c & 3);
    const uint64_t lq0 = (uint64_t)R0 * (uint64_t)a.cols + (uint64_t)(c & ~(int64_t)3);
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = 0u;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const U4 w = sr_words((lq0 + (uint64_t)(i + (int)q) * (uint64_t)a.cols) >> 2, a.seed0_lo,
                            a.seed0_hi);
      const uint32_t own = pick_word(w, q);
      const uint32_t g1 =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 1u), 0xB1, 0xF, 0xF, false);
      const uint32_t g2 =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 2u), 0x4E, 0xF, 0xF, false);
      const uint32_t g3 =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 3u), 0x1B, 0xF, 0xF, false);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t d = (uint32_t)r ^ q;             // row i + r came from lane q ^ d
        uint32_t u = own;
        u = d == 1u ? g1 : u;
        u = d == 2u ? g2 : u;
        u = d == 3u ? g3 : u;
        const uint32_t t = f_bits(__fmul_rn(__fmul_rn(y[i + r], m1), m2));
        out[(i + r) >> 3] |= (e2m1_sr_mag(t & 0x7FFFFFFFu, u >> 8) | ((t >> 28) & 8u))
                             << (4 * ((i + r) & 7));
      }
    }
    if (s == 0xFFu) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) out[j] = 0u;
    }
    return s;
  } else {
    auto u24_of = [](int) -> uint32_t { return 0u; };   // nearest rounding draws nothing
    return quantize_block<RotKind<ROT>::value, RND, FMT>(y, out, u24_of);
  }
}

// A block's codes at p: 16 bytes, or E4M3's two 16-element chunks. ONCE: past
// the caches.
template <bool ONCE, int kWords>
__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t (&out)[kWords]) {
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i) {
    const row_u32x4 v = {out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]};
    row_u32x4 *q = reinterpret_cast<row_u32x4 *>(p + 256 * i);
    if constexpr (ONCE)
      __builtin_nontemporal_store(v, q);
    else
      *q = v;
  }
}

// Whether x, the residual and h together fill three quarters of the 256 MB
// Infinity cache, and are then read around it: see the two launchers for both
// sides' times.
inline bool norm_once(const NormArgs &a) {
  return a.rows * a.cols * (a.f32 ? 4 : 2) * (a.residual ? 3 : 1) >= (int64_t)192 << 20;
}

// One launcher per element format, rounding and rotation.
template <template <int, int, int> class L>
hipError_t norm_dispatch(const NormArgs &a, hipStream_t stream) {
  if (a.fmt == 1) {                       // E4M3: nearest rounding only
    if (a.round != MX_K_ROUND_RNE) return hipErrorInvalidValue;
    switch (a.rotate) {
      case 0: return L<0, 0, kFmtE4M3>::run(a, stream);
      case 1: return L<1, 0, kFmtE4M3>::run(a, stream);
      case 2: return L<2, 0, kFmtE4M3>::run(a, stream);
      case 3: return L<3, 0, kFmtE4M3>::run(a, stream);
      default: return hipErrorInvalidValue;
    }
  }
  if (a.fmt != 0) return hipErrorInvalidValue;
  switch (a.rotate * 2 + a.round) {
    case 0: return L<0, 0, kFmtE2M1>::run(a, stream);
    case 1: return L<0, 1, kFmtE2M1>::run(a, stream);
    case 2: return L<1, 0, kFmtE2M1>::run(a, stream);
    case 3: return L<1, 1, kFmtE2M1>::run(a, stream);
    case 4: return L<2, 0, kFmtE2M1>::run(a, stream);
    case 5: return L<2, 1, kFmtE2M1>::run(a, stream);
    case 6: return L<3, 0, kFmtE2M1>::run(a, stream);
    case 7: return L<3, 1, kFmtE2M1>::run(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mx
