// RMS norm into packed operands for gfx950:
//
//   h = x + residual            rounded to the rows' type, the stream's own
//   rstd = fl32(1 / sqrt(mean_k h_k^2 + eps))
//   y_k = fl32(fl32(h_k * rstd) * weight_k)
//
// and y rotated, scaled and rounded per 32-element block by the quantizers' own
// encoder (mx_encode.h; see encode_row_block for the one difference that y's
// bits make, at values below 2^-126), along the rows (the axis-1 operand of the
// forward product) and, for training, also down the columns (the axis-0
// operand of the weight gradient). y itself is never rounded to bf16 and
// never leaves the chip.
//
// The sum of squares and rstd are held in 64 bits and rounded once: a code or
// a block scale next to a border then depends on y's definition alone, not on
// the order of a sum, and operands can be compared bit for bit. The two
// instructions an element costs (convert and fma) are hidden behind its bytes:
// with fp32 in their place 51.6 us became 51.3 us (8192 x 4096, an earlier
// step).
//
// 8192 x 4096 bf16 with residual, H32, E4M3: 44.4 to 46.3 us (two boxes) for
// 239 MB, 5.2 to 5.4 TB/s, a device copy's rate: bound by HBM. A wave issues 864
// vector instructions for its 2048 elements, half of what fits into that time.
// MXFP4 42.8 us; with stochastic rounding 61.6 us, bound by vector issue (eight
// Philox calls a block: 1763 instructions a wave). One row: 4.6 to 5.0 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "mx_norm_device.h"

namespace mx {

namespace {

// ---------------------------------------------------------------------------
// The axis-1 operand in one pass: a workgroup takes 4 rows, a wave units of 4
// rows x 512 columns (64 blocks, one per lane). Wave w of W holds unit w of h
// in registers, as the rows' type, while the sums of squares meet in LDS; the
// units from W on (rows wider than W of them) are read again, from cache, by
// the lanes that wrote them. Each unit's y then goes through LDS as fp32, from
// the lanes that loaded it (8 columns of each row) to those that encode it
// (lane l: row l % 4, block l / 4).
// Four rows: with eight a compute unit held fewer workgroups to overlap
// (8192 x 4096 50.7 us, against 49.7 us with four, 55 us with two and 74 us
// with one, whose codes are stored 16 bytes at a time; before the weights were
// read ahead). A wave holds one unit: with two, spills (82 us).
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
  // A lane's 8 columns of a unit: 8 that follow each other (bf16) or two times 4,
  // 256 columns apart (fp32), so that in either type one load or store of the
  // wave covers 1 KB without gaps: 8 that follow each other in fp32 leave every
  // access half of each line, and 8192 x 4096 with residual took 89.1 us instead
  // of 78.6 us (436 MB, 5.5 TB/s).
  constexpr int kParts = F32 ? 2 : 1, kPartCols = 8 / kParts;
  auto part_col = [&](uint32_t u, int n) {
    return (int64_t)u * kUnitCols + n * (kUnitCols / kParts) + lane * kPartCols;
  };
  // Columns past the last, which only padding sees: fp32 takes zeros by a branch
  // in each load (a lane may be past with its second part alone), bf16 takes
  // zeros by one branch around a unit's first reading (read_unit) and the row's
  // last columns in its second. Each is the faster one for its type: 512 x 4096
  // bf16 6.6 us against 6.9 us by the branch in each load, 8192 x 4096 fp32
  // 78.6 us by it against 89.7 us. (The zeros of read_unit, which keep h from
  // being used without a value, are 0.05 us of the 6.6.)
  auto load_row = [&](const void *p, int64_t row0, uint32_t u, auto once) {
    Row8<F32> v;
#pragma unroll
    for (int n = 0; n < kParts; ++n) {
      const int64_t k = F32 ? part_col(u, n) : min(part_col(u, n), a.cols - kPartCols);
      v.w[n] = row_u32x4{0u, 0u, 0u, 0u};
      if (!F32 || k < a.cols) v.w[n] = load16<F32, decltype(once)::value>(p, row0 + k);
    }
    return v;
  };
  // held (a std::bool_constant): h is not read again here and is written past
  // the caches
  auto read_unit = [&](uint32_t u, Row8<F32>(&v)[4], auto held) {
    if (!F32 && part_col(u, 0) >= a.cols) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j].w[0] = row_u32x4{0u, 0u, 0u, 0u};
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = load_row(a.x, min(r0 + j, a.rows - 1) * a.ldx, u, std::bool_constant<ONCE>{});
    if (a.residual) {
      Row8<F32> t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        t[j] = load_row(a.residual, min(r0 + j, a.rows - 1) * a.ldr, u, std::bool_constant<ONCE>{});
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = add_rows<F32>(v[j], t[j]);
        if (r0 + j < a.rows) {
#pragma unroll
          for (int n = 0; n < kParts; ++n) {
            if (F32 && part_col(u, n) >= a.cols) continue;
            store16<F32, decltype(held)::value>(a.h, (r0 + j) * a.ldh + part_col(u, n), v[j].w[n]);
          }
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
  auto load_weights = [&](uint32_t u) {
    Row8<1> r;                                          // as load_weight_raw: bf16 in w[0]
    if (!F32) return load_weight_raw(a.weight, a.wf32, min(part_col(u, 0), a.cols - 8));
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int64_t k = min(part_col(u, n), a.cols - 4);
      if (a.wf32) {
        r.w[n] = *reinterpret_cast<const row_u32x4 *>(static_cast<const float *>(a.weight) + k);
      } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 b = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(a.weight) + k);
        r.w[0][2 * n] = b.x;
        r.w[0][2 * n + 1] = b.y;
      }
    }
    return r;
  };
  Row8<F32> held[4];
  const Row8<1> w_held = load_weights(wv);
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
      *reinterpret_cast<float4 *>(chunk(j, F32 ? lane : 2 * lane)) =
          make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(chunk(j, F32 ? 64 + lane : 2 * lane + 1)) =
          make_float4(v[4], v[5], v[6], v[7]);
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
    const Row8<1> w = load_weights(u);
    Row8<F32> v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = load_row(a.h, min(r0 + j, a.rows - 1) * a.ldh, u, std::false_type{});
    encode(u, v, w);
  }
}

// Rows that outgrow the caches (norm_once) are read past them: 8192 x 4096
// 49.8 -> 46.9 us; fewer may be there from what wrote them. Up to 4096 columns
// a workgroup asks for the LDS of eight waves, so that two share a compute
// unit (8192 x 4096 46.4 us, with sixteen waves' LDS 54.7 us); wider rows need
// sixteen.
template <int ROT, int RND, int FMT>
struct Axis1Launch {
  template <int F32, bool ONCE>
  static hipError_t one(const NormArgs &a, hipStream_t stream) {
    const int64_t mnp = (a.rows + 255) & ~(int64_t)255;
    const int waves = (int)std::min<int64_t>(16, (a.cols + kUnitCols - 1) / kUnitCols);
    const dim3 grid((unsigned)(mnp / kRows)), block(waves * 64);
    return waves <= 8
               ? launch(norm_axis1_kernel<F32, ROT, RND, FMT, ONCE, 8>, grid, block, 0, stream, a)
               : launch(norm_axis1_kernel<F32, ROT, RND, FMT, ONCE, 16>, grid, block, 0, stream, a);
  }
  static hipError_t run(const NormArgs &a, hipStream_t stream) {
    const bool once = norm_once(a);
    if (a.f32) return once ? one<1, true>(a, stream) : one<1, false>(a, stream);
    return once ? one<0, true>(a, stream) : one<0, false>(a, stream);
  }
};

}  // namespace

hipError_t norm_launch(const NormArgs &a, hipStream_t stream) {
  return a.codes0 != nullptr ? norm_dual_launch(a, stream) : norm_dispatch<Axis1Launch>(a, stream);
}

}  // namespace mx
