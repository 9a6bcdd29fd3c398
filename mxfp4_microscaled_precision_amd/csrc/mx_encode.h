// Block encoder shared by the quantizers and the norm: rotation, block scale,
// element rounding and the tiled operand layout.
//
// Per 32-element block (36Kr article "Neue Studie von AMD durchbricht die
// bestehende Erkenntnis ...", sections "Was ist MXFP4?" and
// "Fehlerdiagnoseexperiment"): butterfly, amax, E8M0 exponent, E2M1 or E4M3
// elements. One lane holds a whole block in registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mx {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Unnormalised butterfly: h = H32 x in fp32, strides 1, 2, 4, 8, 16, lower
// index a + b, upper a - b. The normalisation y = fl32(h * c) is folded into
// the scale multiply of quantize_block.
__device__ __forceinline__ void butterfly32(float (&y)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if ((i & h) == 0) {
        const float a = y[i];
        const float b = y[i + h];
        y[i] = __fadd_rn(a, b);
        y[i + h] = __fsub_rn(a, b);
      }
    }
  }
}

// The 16-point variant: two independent butterflies (strides 1, 2, 4, 8) on
// elements 0..15 and 16..31; its normalisation 1/4 is applied like c below.
__device__ __forceinline__ void butterfly16x2(float (&y)[32]) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if ((i & h) == 0) {
        const float a = y[i];
        const float b = y[i + h];
        y[i] = __fadd_rn(a, b);
        y[i + h] = __fsub_rn(a, b);
      }
    }
  }
}

typedef short v2i16 __attribute__((ext_vector_type(2)));

// |t| clamped to 448, E4M3's largest finite value (one v_med3_f32).
__device__ __forceinline__ float sat448(float t) {
  return __builtin_amdgcn_fmed3f(t, -448.0f, 448.0f);
}

// Element formats: the E2M1 elements of MXFP4, and the E4M3 elements of the
// MXFP8 comparator (same 32-element blocks and E8M0 scales; one code byte per
// element; nearest-even rounding only).
constexpr int kFmtE2M1 = 0;
constexpr int kFmtE4M3 = 1;

// Rotation kind of the encoder: 0 none, 1 the 32-point Hadamard (with or
// without random signs), 2 the 16-point variant.
template <int ROT>
struct RotKind {
  static constexpr int value = ROT == MX_K_ROT_NONE ? 0 : (ROT == MX_K_ROT_HADAMARD16 ? 2 : 1);
};

template <int ROT>
__device__ __forceinline__ void rotate_block(float (&y)[32]) {
  if (ROT == MX_K_ROT_HADAMARD16)
    butterfly16x2(y);
  else if (ROT != MX_K_ROT_NONE)
    butterfly32(y);
}

// Normalisation of the rotation: fp32(1/sqrt 32), or 1/4 for the 16-point
// variant.
template <int RK>
__device__ __forceinline__ float rot_norm() {
  return RK == 2 ? 0.25f : bits_f(kInvSqrt32Bits);
}

// max |v| of a block after the 32-point rotation, as bits: one v_maximum3_f32
// for two elements, which keeps a NaN where v_max3_f32 skips it. A source block
// that holds a NaN or Inf leaves no output finite, but one of finite values
// whose sums overflow to both infinities can leave NaN beside finite outputs
// and no Inf.
__device__ __forceinline__ uint32_t rotated_amax(const float (&v)[32]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 31; i += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(v[i])),
                                      fabsf(v[i + 1]));
  return f_bits(__builtin_elementwise_maximum(m, fabsf(v[31]))) & 0x7FFFFFFFu;
}

// Quantize one 32-element block. v holds the butterfly output h (RK != 0) or
// the input x (RK == 0). The rotated value is y = fl32(h * c) with c the
// normalisation (rot_norm).
//
//  * amax: max |y| = fl32(max |h| * c), since rounding is monotonic; a NaN
//    or Inf anywhere in the block marks it (see the amax comment below).
//  * scale: e from amax; t = fl32(y * 2^-e). Stochastic rounding reads
//    every bit of t, so it takes the two multiplies as written. For nearest
//    rounding with e <= 123, c_e = c * 2^-e is an exact normal fp32 number
//    and t = fl32(h * c_e) gives the same code as fl32(y * 2^-e): a
//    power-of-two scaling commutes with rounding unless y or t is subnormal.
//    A subnormal t encodes as a signed zero either way. A subnormal y needs
//    |h| < 2^-123.5, and h is then n * 2^-133 with n < 724 (bf16's finest
//    step; butterfly sums of such values are exact); no such n * c comes
//    within fp32 rounding distance of a decision threshold times 2^e (the
//    thresholds are multiples of 2^-10: it would need |16 c n - j| < 2^-13
//    for an integer j, and over n < 724 the closest approach is 8.8e-4, at
//    n = 204).
//    For e > 123 the two multiplies are done as written.
//  * RNE: v_cvt_scalef32_pk_fp4_f32 at scale 1.0, which rounds to nearest
//    even and saturates at +-6 exactly like the threshold rule (checked over
//    every fp32 pattern); two elements per instruction, element 2j in the low
//    nibble. SR: integer rule of e2m1_sr_mag with the Philox uniform. E4M3
//    (nearest only): the hardware fp8 convert behind a clamp to +-448, one
//    code byte per element.
template <int RK, int RND, int FMT, typename U24Fn>
__device__ __forceinline__ uint32_t quantize_block(const float (&v)[32],
                                                   uint32_t (&out)[FMT == kFmtE4M3 ? 8 : 4],
                                                   U24Fn u24_of) {
  constexpr int kWords = FMT == kFmtE4M3 ? 8 : 4;
  // amax as bits of |v| (a NaN or Inf compares above 0x7f800000): integer max
  // of |bits|, or with the 32-point rotation the float max, see rotated_amax.
  uint32_t amax = 0;
  if (RK != 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = max(amax, f_bits(v[i]) & 0x7FFFFFFFu);
  } else {
    amax = rotated_amax(v);
  }
  const bool nonfinite = amax >= 0x7F800000u;
  const float c = rot_norm<RK>();
  if (RK) amax = f_bits(__fmul_rn(bits_f(amax), c));
  // E4M3's largest exponent is 8 where E2M1's is 2: six more below the amax
  const int e = FMT == kFmtE4M3 ? max(block_exponent(amax) - 6, -127) : block_exponent(amax);
  float t[32];
  if (!RK) {
    const float p = pow2_neg(e);
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = __fmul_rn(v[i], p);
  } else if (RND == MX_K_ROUND_SR) {
    const float p = pow2_neg(e);
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = __fmul_rn(__fmul_rn(v[i], c), p);
  } else {
    // c * 2^-e is an exact normal number for e <= 123: one multiply gives
    // the bits of fl32(fl32(h * c) * 2^-e). If some lane of the wave has
    // |y| >= 2^126 (e > 123), the wave multiplies twice: such a lane by c,
    // then by 2^-e, as written; the other lanes by c_e, then by 1, which
    // changes nothing. The first multiply overwrites a copy of v in place,
    // so only one array of 32 is live (a separate array for each case cost
    // 26 more registers in the dual kernel and one wave per SIMD).
    const float ce = __fmul_rn(c, pow2_neg(min(e, 123)));
    float h[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = v[i];
    float mult = ce;
    if (__builtin_expect(__any(e > 123), 0)) {
      const float m1 = e > 123 ? c : ce;
      mult = e > 123 ? pow2_neg(e) : 1.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) h[i] = __fmul_rn(h[i], m1);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = __fmul_rn(h[i], mult);
  }
  if constexpr (FMT == kFmtE4M3) {
    // v_cvt_scalef32_pk_fp8_f32 at scale 1.0 rounds to the nearest E4M3
    // value, ties to even, exactly like the integer rule below 464 (checked
    // over every fp32 value of magnitude below 512) but turns larger
    // magnitudes into NaN; the med3 clamp to +-448 makes it saturate.
    // Element 4j + i goes to byte i of word j.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v2i16 w = {0, 0};
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, sat448(t[4 * j]), sat448(t[4 * j + 1]),
                                                   1.0f, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, sat448(t[4 * j + 2]),
                                                   sat448(t[4 * j + 3]), 1.0f, true);
      out[j] = (uint32_t)(uint16_t)w[0] | ((uint32_t)(uint16_t)w[1] << 16);
    }
  } else if (RND == MX_K_ROUND_SR) {
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t tb = f_bits(t[i]);
      const uint32_t code = e2m1_sr_mag(tb & 0x7FFFFFFFu, u24_of(i)) | ((tb >> 28) & 8u);
      out[i >> 3] |= code << (4 * (i & 7));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w = 0u;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[8 * j + 0], t[8 * j + 1], 1.0f, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[8 * j + 2], t[8 * j + 3], 1.0f, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[8 * j + 4], t[8 * j + 5], 1.0f, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[8 * j + 6], t[8 * j + 7], 1.0f, 3);
      out[j] = w;
    }
  }
  if (nonfinite) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = 0u;
    return 0xFFu;
  }
  return (uint32_t)(e + 127);
}

// Scale of one block for stochastic rounding, t = fl32(fl32(v * m1) * m2):
// m1 = c, m2 = 2^-e with rotation (the two roundings as defined, see
// quantize_block); m1 = 2^-e, m2 = 1 without. Returns the scale code (0xFF
// for a block holding a NaN or Inf, detected as in quantize_block).
template <int RK>
__device__ __forceinline__ uint32_t block_scale(const float (&v)[32], float &m1, float &m2) {
  uint32_t amax = 0;
  if (RK != 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = max(amax, f_bits(v[i]) & 0x7FFFFFFFu);
  } else {
    amax = rotated_amax(v);
  }
  const bool nonfinite = amax >= 0x7F800000u;
  const float c = rot_norm<RK>();
  if (RK) amax = f_bits(__fmul_rn(bits_f(amax), c));
  const int e = block_exponent(amax);
  if (!RK) {
    m1 = pow2_neg(e);
    m2 = 1.0f;
  } else {
    m1 = c;
    m2 = pow2_neg(e);
  }
  return nonfinite ? 0xFFu : (uint32_t)(e + 127);
}

// Sign bits of K indices 4 ctr .. 4 ctr + 3 as a nibble (bit j for index
// 4 ctr + j), from one Philox call of the sign stream.
__device__ __forceinline__ uint32_t sign_nibble(uint32_t ctr, uint32_t seed_lo) {
  const U4 sw = sign_words(ctr, seed_lo);
  return (sw.x >> 31) | ((sw.y >> 31) << 1) | ((sw.z >> 31) << 2) | ((sw.w >> 31) << 3);
}

// The 32 sign bits whose nibbles lanes base .. base + 7 of the wave hold
// (bit i for element i of the block).
__device__ __forceinline__ uint32_t gather_sign_mask(uint32_t nib, int base) {
  uint32_t mask = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) mask |= (uint32_t)__builtin_amdgcn_readlane((int)nib, base + j) << (4 * j);
  return mask;
}

__device__ __forceinline__ void apply_sign_mask(float (&y)[32], uint32_t mask) {
#pragma unroll
  for (int i = 0; i < 32; ++i) y[i] = bits_f(f_bits(y[i]) ^ ((mask << (31 - i)) & 0x80000000u));
}

// ---------------------------------------------------------------------------
// Output layout (tiled, see mx_qtensor in mxfp4.h): the operand is viewed
// reduction-major, [MN, K], zero-padded to [MNp, Kp] (MNp multiple of 256, Kp
// of 128). Codes: tile (g, q) = rows 16g.., K elements 128q.. is 1 KB at
// (g * Kp/128 + q) * 1024, block c of row r at c * 256 + r * 16 inside it.
// Scales: [Kp/128][MNp/256][4][4][16][4], the scale of row 256T + 16h + r,
// block 4q + c at (q * MNp/256 + T) * 1024 + (h / 4) * 256 + c * 64 + r * 4 +
// h % 4. Padding positions hold the encoding of zeros (codes 0, scale code 0).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t code_offset(int64_t mn, int64_t kb, int64_t nslices) {
  return ((mn >> 4) * nslices + (kb >> 2)) * 1024 + (kb & 3) * 256 + (mn & 15) * 16;
}
// E4M3 codes (one byte per element): tile (g, q) is 2 KB at
// (g * Kp/128 + q) * 2048; inside it the 16-element chunk j of row r is the
// 16 bytes at j * 256 + r * 16. Block kb of row mn is chunks 2 (kb % 4) and
// 2 (kb % 4) + 1; this returns the first one's address (the second is 256
// bytes on).
__device__ __forceinline__ int64_t code_offset_e4m3(int64_t mn, int64_t kb, int64_t nslices) {
  return ((mn >> 4) * nslices + (kb >> 2)) * 2048 + (kb & 3) * 512 + (mn & 15) * 16;
}
__device__ __forceinline__ int64_t scale_offset(int64_t mn, int64_t kb, int64_t mnp) {
  const int64_t h = (mn >> 4) & 15;
  return ((kb >> 2) * (mnp >> 8) + (mn >> 8)) * 1024 + (h >> 2) * 256 + (kb & 3) * 64 +
         (mn & 15) * 4 + (h & 3);
}

}  // namespace mx
