// RMS norm into both packed operands of y for gfx950 (see mx_norm.hip for the
// formulas): the axis-0 blocks run down 32 rows, whose rstd has to be known
// first, and 32 whole rows are more than a workgroup can hold next to the
// encoder's registers (a kernel of 16 waves that held them spilled 80
// registers a lane and took 177 us at 16384 x 4096, against 137 us for the two
// launches at the time). So one launch writes h and rstd, and a second reads h
// back, from the Infinity cache, and encodes it both ways. (Encoding the axis-1
// operand in the first launch has not been measured.)
//
// 16384 x 4096 bf16 with residual, H32, E4M3: 61.6 us for the rows (403 MB,
// 6.5 TB/s: bound by memory) and 44.2 us for the pieces, bound by vector issue
// (430 instructions a wave, issued during the whole launch). 4096 x 4096 MXFP4:
// 33.6 us, with stochastic rounding 60.0 us, bound by vector issue. Both in one
// launch, the pieces a slab of rows behind, gained nothing (135 against
// 137 us at the time).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_norm_device.h"

namespace mx {

namespace {

// ---------------------------------------------------------------------------
// h and rstd of every row: a workgroup per row. ONCE: x and the residual are
// kept out of the Infinity cache, so that h is still there when the pieces
// below read it.
// ---------------------------------------------------------------------------
template <int F32, bool ONCE>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs a) {
  const int64_t r = blockIdx.x;
  double acc = 0.0;
  // A thread's 8 columns: adjacent ones (bf16) or two times 4, 1024 apart
  // (fp32), so that each access of a wave covers whole lines (both launches at
  // 8192 x 4096 fp32: 96.7 us, by 8 adjacent columns 108.2 us).
  constexpr int kParts = F32 ? 2 : 1, kPartCols = 8 / kParts;
  auto load = [&](const void *p, int64_t row0, const int64_t (&c)[kParts]) {
    Row8<F32> v;
#pragma unroll
    for (int n = 0; n < kParts; ++n) {
      v.w[n] = row_u32x4{0u, 0u, 0u, 0u};
      if (n == 0 || c[n] < a.cols) v.w[n] = load16<F32, ONCE>(p, row0 + c[n]);
    }
    return v;
  };
  for (int64_t c0 = threadIdx.x * kPartCols; c0 < a.cols; c0 += 256 * 8) {
    int64_t c[kParts];
#pragma unroll
    for (int n = 0; n < kParts; ++n) c[n] = c0 + n * 256 * kPartCols;
    Row8<F32> v = load(a.x, r * a.ldx, c);
    if (a.residual) {
      v = add_rows<F32>(v, load(a.residual, r * a.ldr, c));
#pragma unroll
      for (int n = 0; n < kParts; ++n)
        if (n == 0 || c[n] < a.cols) store16<F32, false>(a.h, r * a.ldh + c[n], v.w[n]);
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

// ---------------------------------------------------------------------------
// Both operands from h and rstd (rows % 32 == 0): a workgroup stages y of 32
// rows x 128 columns in LDS (fp32, row stride 132 floats), then threads
// 0..127 encode its 128 row blocks and threads 128..255 its 128 column blocks.
// ---------------------------------------------------------------------------
template <int F32, int ROT, int RND, int FMT, bool ONCE>
__global__ __launch_bounds__(256) void norm_dual_kernel(NormArgs a, uint32_t gx) {
  __shared__ __attribute__((aligned(16))) float st[32 * 132];
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t by = blockIdx.x / gx, bx = blockIdx.x - by * gx;
  const int64_t C0 = (int64_t)bx * 128, R0 = (int64_t)by * 32;
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

// Where the rows outgrow the Infinity cache (norm_once) x and the residual are
// read around it, so that h is still there for the second launch, and that
// launch's codes are written around it: 16384 x 4096 129.5 -> 115.5 us. With
// less the rows may be there from what wrote them (16384 x 1024: 37.7 us, read
// around the cache 39.5 us), and the codes for the products that read them.
template <int ROT, int RND, int FMT>
struct DualLaunch {
  template <int F32, bool ONCE>
  static hipError_t one(const NormArgs &a, hipStream_t stream) {
    // without a residual h is x and stays
    const dim3 rows((unsigned)a.rows);
    const hipError_t e = ONCE && a.residual
                             ? launch(norm_rows_kernel<F32, true>, rows, dim3(256), 0, stream, a)
                             : launch(norm_rows_kernel<F32, false>, rows, dim3(256), 0, stream, a);
    if (e != hipSuccess) return e;
    // columns up to the axis-0 operand's padded MN extent, rows up to the
    // axis-1 operand's (each covers the other operand's K extent)
    const int64_t gx = ((a.cols + 255) & ~(int64_t)255) / 128;
    const int64_t gy = ((a.rows + 255) & ~(int64_t)255) / 32;
    return launch(norm_dual_kernel<F32, ROT, RND, FMT, ONCE>, dim3((unsigned)(gx * gy)), dim3(256), 0,
                  stream, a, (uint32_t)gx);
  }
  static hipError_t run(const NormArgs &a, hipStream_t stream) {
    const bool once = norm_once(a);
    if (a.f32) return once ? one<1, true>(a, stream) : one<1, false>(a, stream);
    return once ? one<0, true>(a, stream) : one<0, false>(a, stream);
  }
};

}  // namespace

hipError_t norm_dual_launch(const NormArgs &a, hipStream_t stream) {
  return norm_dispatch<DualLaunch>(a, stream);
}

}  // namespace mx
