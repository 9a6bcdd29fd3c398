// RMS norm into packed operands for gfx950:
//
//   h = x + residual            rounded to the rows' type, the stream's own
//   rstd = fl32(1 / sqrt(mean_k h_k^2 + eps))
//   y_k = fl32(fl32(h_k * rstd) * weight_k)
//
// and y rotated, scaled and rounded per 32-element block exactly as the
// quantizers do it (mx_encode.h), along the rows (the axis-1 operand of the
// forward product) and, for training, also down the columns (the axis-0
// operand of the weight gradient). y itself is never rounded to bf16 and
// never leaves the chip.
//
// The sum of squares and rstd are held in 64 bits and rounded once: a code or
// a block scale next to a border then depends on y's definition alone, not on
// the order of a sum, and operands can be compared bit for bit. The two
// instructions an element costs (convert and fma) are hidden behind its
// bytes: the 42 an element of a row may cost before HBM stops being the bound
// are more than twice what the whole kernel issues.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mx_device.h"
#include "mx_encode.h"
#include "mx_kernels.h"
#include "mx_rows.h"

namespace mx {

namespace {


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

// ---------------------------------------------------------------------------
// h and rstd of every row: a workgroup per row. ONCE: x and the residual are
// kept out of the Infinity cache, so that h is still there when the pieces
// below read it.
// ---------------------------------------------------------------------------
template <int F32, bool ONCE>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs a) {
  const int64_t r = blockIdx.x;
  double acc = 0.0;
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += 256 * 8) {
    Row8<F32> v = load8_if<F32, ONCE>(a.x, r * a.ldx + c);
    if (a.residual) {
      v = add_rows<F32>(v, load8_if<F32, ONCE>(a.residual, r * a.ldr + c));
      store8<F32>(a.h, r * a.ldh + c, v);
    }
    float f[8];
    widen8<F32>(v, f);
    acc = add_squares(acc, f);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) acc += __shfl_xor(acc, m);
  __shared__ double part[4];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) a.rstd[r] = rstd_of(part[0] + part[1] + part[2] + part[3], a.inv_cols, a.eps);
}

// The block of y of row r at K = 32 kb of the axis-1 operand, rotated (random
// signs: mask) and rounded; returns its scale code. The stochastic rounding
// index is L = r * cols + 32 kb + i (cols % 32 == 0).
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

// ---------------------------------------------------------------------------
// The axis-1 operand in one pass: a workgroup takes 4 rows, a wave units of 4
// rows x 512 columns (64 blocks, one per lane). Wave w of W holds unit w of h
// in registers, as the rows' type, while the sums of squares meet in LDS; the
// units from W on (rows wider than W of them) are read again, from cache, by
// the lanes that wrote them. Each unit's y then goes through LDS as fp32, from
// the lanes that loaded it (8 columns of each row) to those that encode it
// (lane l: row l % 4, block l / 4).
// ---------------------------------------------------------------------------
constexpr int kRows = 4;
constexpr int kUnitCols = 512;
constexpr int kUnitBlocks = kUnitCols / 32;

__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A double moved between lanes by one DPP control for both halves.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;         // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kDppRor4 = 0x124, kDppRor8 = 0x128;       // row_ror within 16 lanes

// Sums over the wave, four at once: lane l ends up with that of a[l % 4]. In
// two steps a lane hands over what its neighbours keep (three values instead
// of eight), the other four steps move one value.
__device__ __forceinline__ double wave_row_sums(const double (&a)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  const double p = (odd ? a[1] : a[0]) + dpp_f64<kDppXor1>(odd ? a[0] : a[1]);
  const double q = (odd ? a[3] : a[2]) + dpp_f64<kDppXor1>(odd ? a[2] : a[3]);
  double v = (high ? q : p) + dpp_f64<kDppXor2>(high ? p : q);
  v += dpp_f64<kDppRor4>(v);
  v += dpp_f64<kDppRor8>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
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

template <int F32, int ROT, int RND, int FMT, bool ONCE, int MAXW>
__global__ __launch_bounds__(MAXW * 64, 4) void norm_axis1_kernel(NormArgs a) {
  constexpr int kWords = FMT == kFmtE4M3 ? 8 : 4;
  __shared__ __attribute__((aligned(16))) float stage[MAXW][kRows * kUnitCols];
  __shared__ uint8_t signs[ROT == MX_K_ROT_RAND_SIGN ? MAXW : 1][kUnitCols / 4];
  __shared__ double part[MAXW][kRows];
  const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mnp = (a.rows + 255) & ~(int64_t)255;
  const uint32_t nblocks = (uint32_t)((a.cols + 127) >> 7) * 4;      // padding included
  const uint32_t nunits = (nblocks + kUnitBlocks - 1) / kUnitBlocks;
  const int64_t r0 = (int64_t)blockIdx.x * kRows;
  // this lane's row and block of a unit, and where its codes and scales go
  // (below 1 GiB: 32-bit offsets); block kb of a row adds a tile's bytes per
  // slice and a quarter tile per block
  const int er = lane % kRows, eb = lane / kRows;
  const uint32_t m = (uint32_t)(r0 + er);
  const uint32_t codes_row = (m >> 4) * (nblocks * (kWords * 64u)) + (m & 15) * 16u;
  const uint32_t scales_row = (m >> 8) * 1024u + ((m >> 6) & 3) * 256u + (m & 15) * 4u + ((m >> 4) & 3);
  const uint32_t panels = (uint32_t)(mnp >> 8);
  auto put = [&](uint32_t kb, const uint32_t(&out)[kWords], uint32_t s) {
    store_codes<false>(a.codes1 + (codes_row + (kb >> 2) * (kWords * 256u) + (kb & 3) * (kWords * 64u)),
                out);
    a.scales1[scales_row + (kb >> 2) * panels * 1024u + (kb & 3) * 64u] = (uint8_t)s;
  };
  if (r0 >= a.rows) {                                   // padding: zero codes, scale code 0
    uint32_t out[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = 0u;
    for (uint32_t u = wv; u < nunits; u += waves)
      if (u * kUnitBlocks + eb < nblocks) put(u * kUnitBlocks + eb, out, 0u);
    return;
  }
  // a lane loads 8 columns of each row. Rows past the last are read from the
  // last row and not written; columns past the last are not read, and the
  // blocks there are padding.
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  // held (a std::bool_constant): h is not read again here and is written past
  // the caches
  auto read_unit = [&](uint32_t u, Row8<F32>(&v)[4], auto held) {
    const int64_t k = (int64_t)u * kUnitCols + lane * 8;
    if (k >= a.cols) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = load8_if<F32, ONCE>(a.x, min(r0 + j, a.rows - 1) * a.ldx + k);
    if (a.residual) {
      Row8<F32> t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        t[j] = load8_if<F32, ONCE>(a.residual, min(r0 + j, a.rows - 1) * a.ldr + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = add_rows<F32>(v[j], t[j]);
        if (r0 + j < a.rows) {
          if constexpr (decltype(held)::value)
            store8_once<F32>(a.h, (r0 + j) * a.ldh + k, v[j]);
          else
            store8<F32>(a.h, (r0 + j) * a.ldh + k, v[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
      widen8<F32>(v[j], f);
      acc[j] = add_squares(acc[j], f);
    }
  };
  auto column = [&](uint32_t u) { return min((int64_t)u * kUnitCols + lane * 8, a.cols - 8); };
  Row8<F32> held[4];
  const Row8<1> w_held = load_weight_raw(a.weight, a.wf32, column(wv));
  if (wv < (int)nunits) read_unit(wv, held, std::true_type{});
  for (uint32_t u = wv + waves; u < nunits; u += waves) {
    Row8<F32> v[4];
    read_unit(u, v, std::false_type{});
  }

  // row sums over the waves; every wave works out rstd of row l % 4 in lane l
  const double mine = wave_row_sums(acc);
  if (lane < kRows) part[wv][lane] = mine;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < waves; ++i) sum += part[i][er];
  const float rs_er = rstd_of(sum, a.inv_cols, a.eps);
  if (wv == 0 && lane < kRows && r0 + lane < a.rows) a.rstd[r0 + lane] = rs_er;
  float rs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    rs[j] = bits_f((uint32_t)__builtin_amdgcn_readlane((int)f_bits(rs_er), j));

  // The 16-byte chunk c of row r of a unit lies at chunk c ^ f of the row,
  // f = (r + 4 * (c / 16)) % 8, so that the 16 lanes that read a chunk of four
  // rows' four blocks touch distinct banks.
  float *st = stage[wv];
  auto chunk = [&](int r, int c) { return st + r * kUnitCols + ((c ^ ((r + 4 * (c >> 4)) & 7)) << 2); };
  uint8_t *sg = signs[ROT == MX_K_ROT_RAND_SIGN ? wv : 0];
  auto encode = [&](uint32_t u, const Row8<F32>(&h)[4], const Row8<1> &w) {
    wave_lds_sync();                                    // the unit before is read
    float w8[8];
    widen_weight(w, a.wf32, w8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      widen8<F32>(h[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs[j]), w8[i]);
      *reinterpret_cast<float4 *>(chunk(j, 2 * lane)) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(chunk(j, 2 * lane + 1)) = make_float4(v[4], v[5], v[6], v[7]);
    }
    // the unit's reduction indices need kUnitCols / 4 sign calls; the bits meet in
    // LDS as one nibble per call
    if (ROT == MX_K_ROT_RAND_SIGN)
      for (int i = lane; i < kUnitCols / 4; i += 64)
        sg[i] = (uint8_t)sign_nibble(u * (kUnitCols / 4) + i, a.seed1_lo);
    wave_lds_sync();
    const uint32_t kb = u * kUnitBlocks + eb;
    if (kb >= nblocks) return;                          // past the operand's K extent
    float y[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 f = *reinterpret_cast<const float4 *>(chunk(er, eb * 8 + j));
      y[4 * j] = f.x;
      y[4 * j + 1] = f.y;
      y[4 * j + 2] = f.z;
      y[4 * j + 3] = f.w;
    }
    uint32_t mask = 0u;
    if (ROT == MX_K_ROT_RAND_SIGN)
#pragma unroll
      for (int j = 0; j < 8; ++j) mask |= (uint32_t)sg[eb * 8 + j] << (4 * j);
    uint32_t out[kWords];
    uint32_t s = encode_row_block<ROT, RND, FMT>(a, y, r0 + er, kb, mask, out);
    if (r0 + er >= a.rows || ((int64_t)kb << 5) >= a.cols) {   // padding
#pragma unroll
      for (int j = 0; j < kWords; ++j) out[j] = 0u;
      s = 0u;
    }
    put(kb, out, s);
  };
  if (wv < (int)nunits) encode(wv, held, w_held);
  for (uint32_t u = wv + waves; u < nunits; u += waves) {
    const Row8<1> w = load_weight_raw(a.weight, a.wf32, column(u));
    Row8<F32> v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load8<F32>(a.h, min(r0 + j, a.rows - 1) * a.ldh + column(u));
    encode(u, v, w);
  }
}

// ---------------------------------------------------------------------------
// Both operands from h and rstd (rows % 32 == 0): a workgroup stages y of 32
// rows x 128 columns in LDS (fp32, row stride 132 floats), then threads
// 0..127 encode its 128 row blocks and threads 128..255 its 128 column blocks.
// ---------------------------------------------------------------------------
template <int F32, int ROT, int RND, int FMT, bool ONCE>
__global__ __launch_bounds__(256) void norm_dual_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float st[32 * 132];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t C0 = (int64_t)blockIdx.x * 128, R0 = (int64_t)blockIdx.y * 32;
  const int64_t nsl1 = (a.cols + 127) >> 7;   // axis-1 operand: MN = rows, K = cols
  const int64_t nsl0 = (a.rows + 127) >> 7;   // axis-0 operand: MN = cols, K = rows
  const int64_t mnp1 = (a.rows + 255) & ~(int64_t)255, mnp0 = (a.cols + 255) & ~(int64_t)255;
  const bool rows_live = R0 < a.rows;

  if (rows_live) {
    // lane (r0, ch) takes 8 columns of rows r0 and r0 + 16, everything in
    // flight at once; columns past the last are read from the last ones, which
    // only padding sees
    const int ch = tid & 15, r0 = tid >> 4;
    const int64_t c = min(C0 + 8 * ch, a.cols - 8);
    const Row8<1> w = load_weight_raw(a.weight, a.wf32, c);
    Row8<F32> h[2];
    float rs[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) h[j] = load8<F32>(a.h, (R0 + r0 + 16 * j) * a.ldh + c);
#pragma unroll
    for (int j = 0; j < 2; ++j) rs[j] = a.rstd[R0 + r0 + 16 * j];
    float w8[8];
    widen_weight(w, a.wf32, w8);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v[8];
      widen8<F32>(h[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs[j]), w8[i]);
      float *d = st + (r0 + 16 * j) * 132 + 8 * ch;
      *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();

  constexpr int kWords = FMT == kFmtE4M3 ? 8 : 4;
  float y[32];
  uint32_t out[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) out[j] = 0u;
  uint32_t s = 0u;                                        // padding: zero codes, scale code 0
  if (tid < 128) {
    // axis 1: row R0 + rr (< mnp1), 32-block kb along the columns
    const int rr = tid & 31, b = tid >> 5;
    const int64_t r = R0 + rr;
    const int64_t kb = (C0 >> 5) + b;
    uint32_t mask = 0u;
    if (ROT == MX_K_ROT_RAND_SIGN) {
      // this wave's two blocks need the 16 sign calls at counters
      // ((C0 / 32) + 2 wave) * 8 + m, m < 16; lane m makes call m
      const uint32_t nib =
          sign_nibble((uint32_t)(((C0 >> 5) + 2 * (tid >> 6)) * 8 + (lane & 15)), a.seed1_lo);
      const uint32_t m0 = gather_sign_mask(nib, 0), m1 = gather_sign_mask(nib, 8);
      mask = (lane >> 5) ? m1 : m0;
    }
    if (kb >= nsl1 * 4) return;                           // past the operand's K extent
    if ((kb << 5) < a.cols && rows_live) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 f = *reinterpret_cast<const float4 *>(st + rr * 132 + b * 32 + 4 * j);
        y[4 * j] = f.x;
        y[4 * j + 1] = f.y;
        y[4 * j + 2] = f.z;
        y[4 * j + 3] = f.w;
      }
      s = encode_row_block<ROT, RND, FMT>(a, y, r, kb, mask, out);
    }
    store_codes<ONCE>(a.codes1 + (FMT == kFmtE4M3 ? code_offset_e4m3(r, kb, nsl1)
                                            : code_offset(r, kb, nsl1)), out);
    a.scales1[scale_offset(r, kb, mnp1)] = (uint8_t)s;
  } else {
    // axis 0: column C0 + cc (< mnp0), 32-block R0 / 32 along the rows
    const int cc = tid - 128;
    const int64_t c = C0 + cc;
    const int64_t kb = R0 >> 5;
    if (kb >= nsl0 * 4) return;                           // past the operand's K extent (uniform)
    uint32_t mask = 0u;
    if (ROT == MX_K_ROT_RAND_SIGN)   // sign calls R0 / 4 + j; lane j makes call j
      mask = gather_sign_mask(sign_nibble((uint32_t)((R0 >> 2) + (lane & 7)), a.seed0_lo), 0);
    if (rows_live && c < a.cols) {
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = st[j * 132 + cc];
      s = encode_col_block<ROT, RND, FMT>(a, y, R0, c, mask, out);
    }
    store_codes<ONCE>(a.codes0 + (FMT == kFmtE4M3 ? code_offset_e4m3(c, kb, nsl0)
                                            : code_offset(c, kb, nsl0)), out);
    a.scales0[scale_offset(c, kb, mnp0)] = (uint8_t)s;
  }
}

template <int F32, int ROT, int RND, int FMT, bool ONCE>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const int64_t mnp = (a.rows + 255) & ~(int64_t)255;
  if (a.codes0 == nullptr) {
    const int waves = (int)std::min<int64_t>(16, (a.cols + kUnitCols - 1) / kUnitCols);
    const dim3 grid((unsigned)(mnp / kRows)), block(waves * 64);
    return waves <= 8
               ? launch(norm_axis1_kernel<F32, ROT, RND, FMT, ONCE, 8>, grid, block, 0, stream, a)
               : launch(norm_axis1_kernel<F32, ROT, RND, FMT, ONCE, 16>, grid, block, 0, stream, a);
  }
  // without a residual h is x and stays
  const dim3 rows((unsigned)a.rows);
  const hipError_t e = ONCE && a.residual
                           ? launch(norm_rows_kernel<F32, true>, rows, dim3(256), 0, stream, a)
                           : launch(norm_rows_kernel<F32, false>, rows, dim3(256), 0, stream, a);
  if (e != hipSuccess) return e;
  // columns up to the axis-0 operand's padded MN extent, rows up to the axis-1
  // operand's (each covers the other operand's K extent)
  const int64_t gx = ((a.cols + 255) & ~(int64_t)255) / 128;
  return launch(norm_dual_kernel<F32, ROT, RND, FMT, ONCE>,
                dim3((unsigned)gx, (unsigned)(mnp / 32)), dim3(256), 0, stream, a);
}

template <int ROT, int RND, int FMT>
hipError_t launch_norm_type(const NormArgs &a, hipStream_t stream) {
  // Once x, the residual and h together fill three quarters of the 256 MB
  // Infinity cache, x and the residual are read around it, so that h is still
  // there for the second launch of the two-operand pass, and that launch's
  // codes are written around it (16384 x 4096: 129.5 us, with both 115.5 us). In
  // one pass (8192 x 4096) 49.8 -> 46.9 us. With less the rows may be there
  // from what wrote them (16384 x 1024, two operands: 37.7 us, read around the
  // cache 39.5 us), and the codes for the products that read them.
  const bool once = a.rows * a.cols * (a.f32 ? 4 : 2) * (a.residual ? 3 : 1) >= (int64_t)192 << 20;
  if (a.f32)
    return once ? launch_norm<1, ROT, RND, FMT, true>(a, stream)
                : launch_norm<1, ROT, RND, FMT, false>(a, stream);
  return once ? launch_norm<0, ROT, RND, FMT, true>(a, stream)
              : launch_norm<0, ROT, RND, FMT, false>(a, stream);
}

}  // namespace

hipError_t norm_launch(const NormArgs &a, hipStream_t stream) {
  if (a.fmt == 1) {                       // E4M3: nearest rounding only
    if (a.round != MX_K_ROUND_RNE) return hipErrorInvalidValue;
    switch (a.rotate) {
      case 0: return launch_norm_type<0, 0, kFmtE4M3>(a, stream);
      case 1: return launch_norm_type<1, 0, kFmtE4M3>(a, stream);
      case 2: return launch_norm_type<2, 0, kFmtE4M3>(a, stream);
      case 3: return launch_norm_type<3, 0, kFmtE4M3>(a, stream);
      default: return hipErrorInvalidValue;
    }
  }
  if (a.fmt != 0) return hipErrorInvalidValue;
  switch (a.rotate * 2 + a.round) {
    case 0: return launch_norm_type<0, 0, kFmtE2M1>(a, stream);
    case 1: return launch_norm_type<0, 1, kFmtE2M1>(a, stream);
    case 2: return launch_norm_type<1, 0, kFmtE2M1>(a, stream);
    case 3: return launch_norm_type<1, 1, kFmtE2M1>(a, stream);
    case 4: return launch_norm_type<2, 0, kFmtE2M1>(a, stream);
    case 5: return launch_norm_type<2, 1, kFmtE2M1>(a, stream);
    case 6: return launch_norm_type<3, 0, kFmtE2M1>(a, stream);
    case 7: return launch_norm_type<3, 1, kFmtE2M1>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mx
