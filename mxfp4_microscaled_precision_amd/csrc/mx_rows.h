// Row access shared by the norm and its gradient: eight elements of a bf16 or
// fp32 row (16 or 32 bytes) as one unit, adjacent ones or two times four,
// widened to fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

typedef uint32_t row_u32x4 __attribute__((ext_vector_type(4)));

// Eight elements in their type, 16 bytes to a word. F32: fp32 rows, else bf16.
template <int F32>
struct Row8 {
  row_u32x4 w[F32 ? 2 : 1];
};

template <int F32, typename I>
__device__ __forceinline__ Row8<F32> load8(const void *base, I i) {
  Row8<F32> r;
  const row_u32x4 *p = reinterpret_cast<const row_u32x4 *>(
      static_cast<const uint8_t *>(base) + i * (F32 ? 4 : 2));
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) r.w[k] = p[k];
  return r;
}

// 16 bytes of a row from element i on. ONCE: they are not read again soon, so
// the access does not displace what is. It is a template parameter because the
// compiler merges the two sides of a branch and drops the hint.
template <int F32, bool ONCE, typename I>
__device__ __forceinline__ row_u32x4 load16(const void *base, I i) {
  const row_u32x4 *p = reinterpret_cast<const row_u32x4 *>(static_cast<const uint8_t *>(base) +
                                                           i * (F32 ? 4 : 2));
  if constexpr (ONCE)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

template <int F32, bool ONCE, typename I>
__device__ __forceinline__ void store16(void *base, I i, row_u32x4 v) {
  row_u32x4 *p = reinterpret_cast<row_u32x4 *>(static_cast<uint8_t *>(base) + i * (F32 ? 4 : 2));
  if constexpr (ONCE)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

template <int F32, typename I>
__device__ __forceinline__ void store8(void *base, I i, const Row8<F32> &r) {
  row_u32x4 *p = reinterpret_cast<row_u32x4 *>(static_cast<uint8_t *>(base) + i * (F32 ? 4 : 2));
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) p[k] = r.w[k];
}

template <int F32>
__device__ __forceinline__ void widen8(const Row8<F32> &r, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bits_f(r.w[i >> 2][i & 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bits_f(r.w[0][i] << 16);
      v[2 * i + 1] = bits_f(r.w[0][i] & 0xFFFF0000u);
    }
  }
}

// fp32 values as row elements: bf16 rounds to nearest even, one
// v_cvt_pk_bf16_f32 for two.
template <int F32>
__device__ __forceinline__ Row8<F32> narrow8(const float (&v)[8]) {
  Row8<F32> r;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i >> 2][i & 3] = f_bits(v[i]);
  } else {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 p = {v[2 * i], v[2 * i + 1]};
      r.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf2));
    }
  }
  return r;
}

// Eight consecutive weights from index i (i % 8 == 0, 16-byte aligned base).
__device__ __forceinline__ void load_weight8(const void *w, int f32, int64_t i, float (&v)[8]) {
  if (f32)
    widen8<1>(load8<1>(w, i), v);
  else
    widen8<0>(load8<0>(w, i), v);
}

// Four of them.
__device__ __forceinline__ void load_weight4(const void *w, int f32, int64_t i, float *v) {
  if (f32) {
    const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + i);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
    const uint2 b = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(w) + i);
    v[0] = __builtin_bit_cast(float, b.x << 16);
    v[1] = __builtin_bit_cast(float, b.x & 0xFFFF0000u);
    v[2] = __builtin_bit_cast(float, b.y << 16);
    v[3] = __builtin_bit_cast(float, b.y & 0xFFFF0000u);
  }
}

}  // namespace mx
