// Quantizer of rows that belong to groups (one expert's rows after another's),
// gathered on the way: the axis-1 operand of all rows and, from the same read,
// the axis-0 operand in which each group's rows start a 128-deep slice of
// their own, so that no 32-block (its rotation, its scale) holds rows of two
// groups; and the column sums of each group's rows.
//
// Every block is encoded as in mx_quant.hip (see mx_encode.h). A workgroup
// stages 32 rows of one group x 128 columns in LDS as fp32 (row stride 132
// floats: one 16-byte chunk of padding spreads the accesses over the banks).
// Threads 0..127 encode its 128 row blocks for the axis-1 operand; threads
// 128..255 its 128 column blocks for the axis-0 operand, where rows behind the
// group's last are zeros, and add up the columns. Row blocks are written
// wherever their row lies in its 16-row tile: a group may begin at any row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx_encode.h"
#include "mx_groups.h"
#include "mx_kernels.h"

namespace mx {

namespace {

constexpr int kPitch = 132;

// Source row of row r, or -1: without an index r itself; an index outside the
// source gives a row of zeros.
__device__ __forceinline__ int64_t source_row(const GroupedQuantArgs &a, int64_t r) {
  if (!a.index) return r;
  const int64_t i = a.index64 ? static_cast<const int64_t *>(a.index)[r]
                              : static_cast<const int32_t *>(a.index)[r];
  return i >= 0 && i < a.src_rows ? i : -1;
}

template <int ROT, int RND>
__global__ __launch_bounds__(256, 8) void quant_grouped_kernel(GroupedQuantArgs a, uint32_t gx) {
  __shared__ __attribute__((aligned(16))) float st[32 * kPitch];
  const int tid = threadIdx.x, lane = tid & 63;
  const int bx = (int)(blockIdx.x % gx), by = (int)(blockIdx.x / gx);
  const int64_t C0 = (int64_t)bx * 128;
  const int64_t cols = a.cols;
  const int64_t nsl1 = (cols + 127) >> 7, nsl0 = a.slices;
  const int64_t mnp1 = ((int64_t)a.rows + 255) & ~(int64_t)255, mnp0 = (cols + 255) & ~(int64_t)255;

  // 32-deep block `by` of the groups, four to a slice; behind the last group
  // by counts on: zeros for the axis-0 operand's slices that are left, and for
  // the axis-1 operand's rows in no group.
  const Group gr = find_group<true>(a.ends, a.groups, a.rows, a.each, by >> 2, CountSlices());
  const bool in_group = gr.g < a.groups;
  const int step = by - 4 * gr.before;                 // blocks since the group's first
  const int64_t R0 = (int64_t)gr.first + (int64_t)step * 32;
  const int64_t end1 = in_group ? gr.last : mnp1;      // axis-1 rows are written up to here
  const int64_t kb0 = by;                              // axis-0 block along K
  const int live = in_group ? (int)min((int64_t)32, (int64_t)gr.last - R0) : 0;   // rows, <= 0: none

  if (live > 0) {
    // lane (r0, q) loads columns 4q .. and 64 + 4q .. of rows r0 and r0 + 16,
    // all four in flight; rows behind the group's last are zeros
    const int q = tid & 15, r0 = tid >> 4;
    const int64_t c = C0 + 4 * q;
    u32x2 v[4] = {{0u, 0u}, {0u, 0u}, {0u, 0u}, {0u, 0u}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 16 * h;
      const int64_t s = r < live ? source_row(a, R0 + r) : -1;
      if (s >= 0) {
        const uint16_t *p = a.x + s * a.ld + c;
        if (c < cols) v[2 * h] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
        if (c + 64 < cols)
          v[2 * h + 1] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p + 64));
      }
    }
    float *d = st + r0 * kPitch + 4 * q;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<float4 *>(d + (k >> 1) * 16 * kPitch + (k & 1) * 64) =
          make_float4(bits_f(v[k].x << 16), bits_f(v[k].x & 0xFFFF0000u), bits_f(v[k].y << 16),
                      bits_f(v[k].y & 0xFFFF0000u));
  }
  __syncthreads();

  float y[32];
  uint32_t out[4];
  uint32_t s;
  if (tid < 128) {
    // axis 1: row R0 + rr, 32-block kb along the columns
    const int rr = tid & 31, b = tid >> 5;
    const int64_t r = R0 + rr, kb = (C0 >> 5) + b;
    uint32_t mask = 0u;
    if (ROT == MX_K_ROT_RAND_SIGN) {
      // this wave's two blocks: counters ((C0 / 32) + 2 wave) * 8 + m, lane m
      const uint32_t nib =
          sign_nibble((uint32_t)(((C0 >> 5) + 2 * (tid >> 6)) * 8 + (lane & 15)), a.seed1_lo);
      const uint32_t m0 = gather_sign_mask(nib, 0), m1 = gather_sign_mask(nib, 8);
      mask = (lane >> 5) ? m1 : m0;
    }
    if (r >= end1 || kb >= nsl1 * 4) return;
    if (live > 0 && (kb << 5) < cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 f = *reinterpret_cast<const float4 *>(st + rr * kPitch + b * 32 + 4 * j);
        y[4 * j] = f.x;
        y[4 * j + 1] = f.y;
        y[4 * j + 2] = f.z;
        y[4 * j + 3] = f.w;
      }
      if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
      rotate_block<ROT>(y);
      const uint64_t q0 = (uint64_t)(r * cols + (kb << 5)) >> 2;
      U4 w{0u, 0u, 0u, 0u};
      auto u24_of = [&](int i) -> uint32_t {
        if ((i & 3) == 0) w = sr_words(q0 + (uint64_t)(i >> 2), a.seed1_lo, a.seed1_hi);
        return pick_word(w, (uint32_t)(i & 3)) >> 8;
      };
      s = quantize_block<RotKind<ROT>::value, RND, kFmtE2M1>(y, out, u24_of);
    } else {                                           // rows of no group, padding of K
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = 0u;
      s = 0u;
    }
    *reinterpret_cast<uint4 *>(a.codes1 + code_offset(r, kb, nsl1)) =
        make_uint4(out[0], out[1], out[2], out[3]);
    a.scales1[scale_offset(r, kb, mnp1)] = (uint8_t)s;
    return;
  }
  // axis 0: column C0 + cc, block kb0 along the rows
  const int cc = tid - 128;
  const int64_t c = C0 + cc;                           // < mnp0 (grid)
  uint32_t mask = 0u;
  if (ROT == MX_K_ROT_RAND_SIGN)                       // the index within the group's K
    mask = gather_sign_mask(sign_nibble((uint32_t)(step * 8 + (lane & 7)), a.seed0_lo), 0);
  if (live > 0 && c < cols) {                          // uniform over each quad (cols % 32 == 0)
#pragma unroll
    for (int j = 0; j < 32; ++j) y[j] = st[j * kPitch + cc];
    if (a.partial) {
      // the 32 rows' sum, by halves (rows behind the last are zeros)
      float t[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) t[j] = y[j] + y[j + 16];
#pragma unroll
      for (int h = 8; h > 0; h >>= 1)
#pragma unroll
        for (int j = 0; j < h; ++j) t[j] += t[j + h];
      a.partial[(int64_t)by * cols + c] = t[0];
    }
    if (!a.codes0) return;
    if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
    rotate_block<ROT>(y);
    if (RND == MX_K_ROUND_SR) {
      // element (row, c) draws word c % 4 of the call at (row cols + c) / 4;
      // the four lanes of a quad share each call (see quant_axis0_sr_kernel)
      float m1, m2;
      s = block_scale<RotKind<ROT>::value>(y, m1, m2);
      const uint32_t q = (uint32_t)(cc & 3);
      const uint64_t lq0 = (uint64_t)R0 * (uint64_t)cols + (uint64_t)(c & ~(int64_t)3);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = 0u;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const U4 w =
            sr_words((lq0 + (uint64_t)(i + (int)q) * (uint64_t)cols) >> 2, a.seed0_lo, a.seed0_hi);
        const uint32_t own = pick_word(w, q);
        const uint32_t g1 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 1u),
                                                                  0xB1, 0xF, 0xF, false);
        const uint32_t g2 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 2u),
                                                                  0x4E, 0xF, 0xF, false);
        const uint32_t g3 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, q ^ 3u),
                                                                  0x1B, 0xF, 0xF, false);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t d = (uint32_t)r ^ q;
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
        for (int j = 0; j < 4; ++j) out[j] = 0u;
      }
    } else {
      auto u24_of = [](int) -> uint32_t { return 0u; };   // nearest rounding draws nothing
      s = quantize_block<RotKind<ROT>::value, RND, kFmtE2M1>(y, out, u24_of);
    }
  } else {                                             // K padding of the operand
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0u;
    s = 0u;
  }
  if (!a.codes0 || kb0 >= nsl0 * 4) return;
  *reinterpret_cast<uint4 *>(a.codes0 + code_offset(c, kb0, nsl0)) =
      make_uint4(out[0], out[1], out[2], out[3]);
  a.scales0[scale_offset(c, kb0, mnp0)] = (uint8_t)s;
}

// sums[e][c] = the partial sums of group e's blocks. A workgroup has 64 columns
// and four waves that take every fourth block each; their sums meet in LDS.
__global__ __launch_bounds__(256) void group_sums_kernel(GroupedQuantArgs a, uint32_t gx) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (int)(blockIdx.x / gx);
  const int64_t c = (int64_t)(blockIdx.x % gx) * 64 + lane;
  const Group gr = find_group<false>(a.ends, a.groups, a.rows, a.each, e, CountSlices());
  const int blocks = (gr.last - gr.first + 31) >> 5;
  float sum = 0.0f;
  if (c < a.cols) {
    const float *p = a.partial + (int64_t)gr.before * 4 * a.cols + c;
#pragma unroll 4
    for (int b = wave; b < blocks; b += 4) sum += p[(int64_t)b * a.cols];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && c < a.cols)
    a.sums[(int64_t)e * a.cols + c] =
        (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

template <int ROT, int RND>
hipError_t launch_grouped(const GroupedQuantArgs &a, hipStream_t stream) {
  const int64_t gx = ((a.cols + 255) & ~(int64_t)255) / 128;
  // the groups' slices, and behind them whichever is longer of the slices left
  // and the axis-1 operand's rows in no group: 4 slices more hold the latter
  const int64_t gy = 4 * ((int64_t)a.slices + 4);
  if (gx * gy > INT32_MAX) return hipErrorInvalidValue;
  return launch(quant_grouped_kernel<ROT, RND>, dim3((unsigned)(gx * gy)), dim3(256), 0, stream, a,
                (uint32_t)gx);
}

}  // namespace

hipError_t quantize_grouped_launch(const GroupedQuantArgs &a, hipStream_t stream) {
  hipError_t e = hipErrorInvalidValue;
  if (a.rows > 0) {
    switch (a.rotate * 2 + a.round) {
      case 0: e = launch_grouped<0, 0>(a, stream); break;
      case 1: e = launch_grouped<0, 1>(a, stream); break;
      case 2: e = launch_grouped<1, 0>(a, stream); break;
      case 3: e = launch_grouped<1, 1>(a, stream); break;
      case 4: e = launch_grouped<2, 0>(a, stream); break;
      case 5: e = launch_grouped<2, 1>(a, stream); break;
      case 6: e = launch_grouped<3, 0>(a, stream); break;
      case 7: e = launch_grouped<3, 1>(a, stream); break;
    }
    if (e != hipSuccess) return e;
  }
  if (!a.sums) return hipSuccess;
  const int64_t gx = (a.cols + 63) / 64;
  if (gx * a.groups > INT32_MAX) return hipErrorInvalidValue;
  return launch(group_sums_kernel, dim3((unsigned)(gx * a.groups)), dim3(256), 0, stream, a,
                (uint32_t)gx);
}

}  // namespace mx
