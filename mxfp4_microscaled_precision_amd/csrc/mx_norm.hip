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

__device__ __forceinline__ float rstd_of(double sum, int64_t cols, double eps) {
  return (float)(1.0 / __builtin_sqrt(sum / (double)cols + eps));
}

// ---------------------------------------------------------------------------
// h and rstd of every row: a workgroup per row.
// ---------------------------------------------------------------------------
template <int F32>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs a) {
  const int64_t r = blockIdx.x;
  double acc = 0.0;
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += 256 * 8) {
    Row8<F32> v = load8<F32>(a.x, r * a.ldx + c);
    if (a.residual) {
      v = add_rows<F32>(v, load8<F32>(a.residual, r * a.ldr + c));
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
  if (threadIdx.x == 0) a.rstd[r] = rstd_of(part[0] + part[1] + part[2] + part[3], a.cols, a.eps);
}

// ---------------------------------------------------------------------------
// A tile of y (16 rows x 128 columns, fp32) in LDS: the 16-byte chunk c of row
// r lies at r * 512 + (c ^ r) * 16, so that 16 lanes that read one chunk of 16
// rows, or write 16 chunks of one row, touch distinct banks.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float *tile_chunk(float *st, int r, int c) {
  return st + r * 128 + ((c ^ r) << 2);
}

__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Encode the tile (row group g, K slice q) of the axis-1 operand whose y the
// wave has put into st: lane l takes row l % 16, block l / 16.
template <int ROT, int RND, int FMT>
__device__ __forceinline__ void encode_tile(const NormArgs &a, float *st, uint32_t *sg, uint32_t g,
                                            uint32_t q, uint32_t nslices, int64_t mnp) {
  const int lane = threadIdx.x & 63;
  const int rr = lane & 15, cb = lane >> 4;
  const int64_t r = (int64_t)g * 16 + rr;
  const int64_t kb = (int64_t)q * 4 + cb;
  const bool valid = r < a.rows && (kb << 5) < a.cols;
  float y[32];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 f = *reinterpret_cast<const float4 *>(tile_chunk(st, rr, cb * 8 + j));
    y[4 * j] = f.x;
    y[4 * j + 1] = f.y;
    y[4 * j + 2] = f.z;
    y[4 * j + 3] = f.w;
  }
  if (ROT == MX_K_ROT_RAND_SIGN) {
    // the tile's 128 reduction indices need 32 Philox calls: lanes 0..31
    // make one each, the sign bits meet in LDS as one nibble per call
    if (lane < 32) sg[lane] = sign_nibble(q * 32 + lane, a.seed1_lo);
    wave_lds_sync();
    uint32_t mask = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) mask |= sg[cb * 8 + j] << (4 * j);
    apply_sign_mask(y, mask);
  }
  rotate_block<ROT>(y);
  // stochastic rounding index L = r * cols + kb * 32 + i (cols % 32 == 0)
  const uint64_t q0 = (uint64_t)(r * a.cols + (kb << 5)) >> 2;
  U4 w{0u, 0u, 0u, 0u};
  auto u24_of = [&](int i) -> uint32_t {
    if ((i & 3) == 0) w = sr_words(q0 + (uint64_t)(i >> 2), a.seed1_lo, a.seed1_hi);
    return pick_word(w, (uint32_t)(i & 3)) >> 8;
  };
  constexpr int kWords = FMT == kFmtE4M3 ? 8 : 4;
  uint32_t out[kWords];
  uint32_t s = quantize_block<RotKind<ROT>::value, RND, FMT>(y, out, u24_of);
  if (!valid) {                                           // padding: zero codes, scale code 0
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = 0u;
    s = 0u;
  }
  const size_t tile = (size_t)g * nslices + q;
  if constexpr (FMT == kFmtE4M3) {  // block cb of row rr: chunks 2 cb and 2 cb + 1
    uint8_t *tp = a.codes1 + tile * 2048 + cb * 512 + rr * 16;
    *reinterpret_cast<uint4 *>(tp) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint4 *>(tp + 256) = make_uint4(out[4], out[5], out[6], out[7]);
  } else {
    *reinterpret_cast<uint4 *>(a.codes1 + tile * 1024 + lane * 16) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
  a.scales1[scale_offset(r, kb, mnp)] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// The axis-1 operand from h and rstd: a wave per tile, four per workgroup.
// ---------------------------------------------------------------------------
template <int F32, int ROT, int RND, int FMT>
__global__ __launch_bounds__(256) void norm_axis1_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float stage[4][16 * 128];
  __shared__ uint32_t signs[ROT == MX_K_ROT_RAND_SIGN ? 4 : 1][32];
  const int64_t mnp = (a.rows + 255) & ~(int64_t)255;
  const uint32_t nslices = (uint32_t)((a.cols + 127) >> 7);
  const uint32_t ntiles = (uint32_t)(mnp >> 4) * nslices;
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t tile = blockIdx.x * 4u + (uint32_t)wv;
  if (tile >= ntiles) return;
  const uint32_t g = tile / nslices, q = tile - g * nslices;
  float *st = stage[wv];
  // lane l takes 8 columns of row 4 j + l / 16. Rows and columns past the
  // source are read from its last row and last chunk: only padding uses them.
  const int ch = lane & 15;
  const int64_t k = min((int64_t)q * 128 + ch * 8, a.cols - 8);
  float w8[8];
  load_weight8(a.weight, a.wf32, k, w8);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int rr = j * 4 + (lane >> 4);
    const int64_t r = min((int64_t)g * 16 + rr, a.rows - 1);
    float v[8];
    widen8<F32>(load8<F32>(a.h, r * a.ldh + k), v);
    const float rs = a.rstd[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs), w8[i]);
    *reinterpret_cast<float4 *>(tile_chunk(st, rr, 2 * ch)) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(tile_chunk(st, rr, 2 * ch + 1)) =
        make_float4(v[4], v[5], v[6], v[7]);
  }
  wave_lds_sync();
  encode_tile<ROT, RND, FMT>(a, st, signs[ROT == MX_K_ROT_RAND_SIGN ? wv : 0], g, q, nslices, mnp);
}

// ---------------------------------------------------------------------------
// Both operands from h and rstd (rows % 32 == 0): a workgroup stages y of 32
// rows x 128 columns in LDS (fp32, row stride 132 floats), then threads
// 0..127 encode its 128 row blocks and threads 128..255 its 128 column blocks.
// ---------------------------------------------------------------------------
template <int F32, int ROT, int RND, int FMT>
__global__ __launch_bounds__(256) void norm_dual_kernel(NormArgs a, int64_t gx) {
  __shared__ __attribute__((aligned(16))) float st[32 * 132];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t bx = (int64_t)blockIdx.x % gx, by = (int64_t)blockIdx.x / gx;
  const int64_t C0 = bx * 128, R0 = by * 32;
  const int64_t nsl1 = (a.cols + 127) >> 7;   // axis-1 operand: MN = rows, K = cols
  const int64_t nsl0 = (a.rows + 127) >> 7;   // axis-0 operand: MN = cols, K = rows
  const int64_t mnp1 = (a.rows + 255) & ~(int64_t)255, mnp0 = (a.cols + 255) & ~(int64_t)255;
  const bool rows_live = R0 < a.rows;

  if (rows_live) {
    // lane (r0, ch) takes 8 columns of rows r0 and r0 + 16
    const int ch = tid & 15, r0 = tid >> 4;
    const int64_t c = C0 + 8 * ch;
    float w8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < a.cols) load_weight8(a.weight, a.wf32, c, w8);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int rr = r0 + 16 * j;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (c < a.cols) {
        widen8<F32>(load8<F32>(a.h, (R0 + rr) * a.ldh + c), v);
        const float rs = a.rstd[R0 + rr];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs), w8[i]);
      }
      float *d = st + rr * 132 + 8 * ch;
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
  U4 w{0u, 0u, 0u, 0u};
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
      if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
      rotate_block<ROT>(y);
      const uint64_t q0 = (uint64_t)(r * a.cols + (kb << 5)) >> 2;   // L % 4 == 0
      auto u24_of = [&](int i) -> uint32_t {
        if ((i & 3) == 0) w = sr_words(q0 + (uint64_t)(i >> 2), a.seed1_lo, a.seed1_hi);
        return pick_word(w, (uint32_t)(i & 3)) >> 8;
      };
      s = quantize_block<RotKind<ROT>::value, RND, FMT>(y, out, u24_of);
    }
    if constexpr (FMT == kFmtE4M3) {
      uint8_t *p = a.codes1 + code_offset_e4m3(r, kb, nsl1);
      *reinterpret_cast<uint4 *>(p) = make_uint4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<uint4 *>(p + 256) = make_uint4(out[4], out[5], out[6], out[7]);
    } else {
      *reinterpret_cast<uint4 *>(a.codes1 + code_offset(r, kb, nsl1)) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
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
      if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
      rotate_block<ROT>(y);
      // element (R0 + i, c) has L = (R0 + i) cols + c
      auto u24_of = [&](int i) -> uint32_t {
        const uint64_t L = (uint64_t)((R0 + i) * a.cols + c);
        return pick_word(sr_words(L >> 2, a.seed0_lo, a.seed0_hi), (uint32_t)(L & 3)) >> 8;
      };
      s = quantize_block<RotKind<ROT>::value, RND, FMT>(y, out, u24_of);
    }
    if constexpr (FMT == kFmtE4M3) {
      uint8_t *p = a.codes0 + code_offset_e4m3(c, kb, nsl0);
      *reinterpret_cast<uint4 *>(p) = make_uint4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<uint4 *>(p + 256) = make_uint4(out[4], out[5], out[6], out[7]);
    } else {
      *reinterpret_cast<uint4 *>(a.codes0 + code_offset(c, kb, nsl0)) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
    a.scales0[scale_offset(c, kb, mnp0)] = (uint8_t)s;
  }
}

template <int F32, int ROT, int RND, int FMT>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const hipError_t e =
      launch(norm_rows_kernel<F32>, dim3((unsigned)a.rows), dim3(256), 0, stream, a);
  if (e != hipSuccess) return e;
  const int64_t mnp = (a.rows + 255) & ~(int64_t)255;
  if (a.codes0 == nullptr) {
    const int64_t ntiles = (mnp >> 4) * ((a.cols + 127) >> 7);
    return launch(norm_axis1_kernel<F32, ROT, RND, FMT>, dim3((unsigned)((ntiles + 3) / 4)),
                  dim3(256), 0, stream, a);
  }
  // columns up to the axis-0 operand's padded MN extent, rows up to the axis-1
  // operand's (each covers the other operand's K extent)
  const int64_t gx = ((a.cols + 255) & ~(int64_t)255) / 128;
  const int64_t gy = mnp / 32;
  return launch(norm_dual_kernel<F32, ROT, RND, FMT>, dim3((unsigned)(gx * gy)), dim3(256), 0,
                stream, a, gx);
}

template <int ROT, int RND, int FMT>
hipError_t launch_norm_type(const NormArgs &a, hipStream_t stream) {
  return a.f32 ? launch_norm<1, ROT, RND, FMT>(a, stream) : launch_norm<0, ROT, RND, FMT>(a, stream);
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
