// Quantizer of rows that belong to groups (one expert's rows after another's),
// gathered on the way: the axis-1 operand of all rows and, from the same read,
// the axis-0 operand in which each group's rows start a 128-deep slice of
// their own, so that no 32-block (its rotation, its scale) holds rows of two
// groups; and the column sums of each group's rows.
//
// Every block is encoded as in mx_quant.hip (see mx_encode.h). A workgroup has a
// slice, 128 rows of one group, x 128 columns. It stages 32 rows at a time in LDS as
// fp32 (row stride 132 floats: one 16-byte chunk of padding spreads the accesses
// over the banks) while the next 32 are on their way in registers. Threads 0..127
// encode the 128 row blocks for the axis-1 operand; threads 128..255 the 128 column
// blocks for the axis-0 operand, where rows behind the group's last are zeros, and
// add up the columns. Row blocks are written wherever their row lies in its 16-row
// tile: a group may begin at any row. The group is looked up once for a slice: once
// for 32 rows, in four times as many workgroups, the look-up stood before every
// load (16384x4096, 8 groups: 58.7 us, now 53.7; through an index 58.7).
//
// Bound by vector issue where there are many rows, as the ordinary two-operand
// quantizer (40.4 us there). 16384x4096 through an index takes 59 us; by counters a
// wave issues 1376 vector instructions, and the SIMDs do so in 81% of the cycles that
// the kernel is busy. It moves 206 MB in that time, 3.5 TB/s, of which a row that the
// index names twice is read once from memory. The ordinary one encodes a row block and
// a column block with all 256 threads; here a group's last slice has rows of none, and
// row blocks begin at any row of a tile. 8 waves a SIMD instead of 4 spill (91 us).
// Small calls wait as long as they issue: 8192x1056 of 64 experts without a rotation,
// 12.6 us, 59%, in 1.3 rounds of workgroups.
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

// y[LO] + .. + y[LO + N - 1], by halves.
template <int LO, int N>
__device__ __forceinline__ float sum_of(const float (&y)[32]) {
  if constexpr (N == 1)
    return y[LO];
  else
    return sum_of<LO, N / 2>(y) + sum_of<LO + N / 2, N / 2>(y);
}

template <int ROT, int RND>
__global__ __launch_bounds__(256, 4) void quant_grouped_kernel(GroupedQuantArgs a, uint32_t gx) {
  __shared__ __attribute__((aligned(16))) float st[32 * kPitch];
  const int tid = threadIdx.x, lane = tid & 63;
  const int bx = (int)(blockIdx.x % gx), by = (int)(blockIdx.x / gx);
  const int64_t C0 = (int64_t)bx * 128;
  const int64_t cols = a.cols;
  const int64_t nsl1 = (cols + 127) >> 7, nsl0 = a.slices;
  const int64_t mnp1 = ((int64_t)a.rows + 255) & ~(int64_t)255, mnp0 = (cols + 255) & ~(int64_t)255;

  // Slice `by` of the groups; behind the last group by counts on: zeros for the
  // axis-0 operand's slices that are left, and for the axis-1 operand's rows in
  // no group.
  const Group gr = find_group<true>(a.ends, a.groups, a.rows, a.each, by, CountSlices());
  const bool in_group = gr.g < a.groups;
  const int64_t S0 = (int64_t)gr.first + (int64_t)(by - gr.before) * 128;   // the slice's first row
  const int64_t end1 = in_group ? gr.last : mnp1;      // axis-1 rows are written up to here
  const int rows = in_group ? (int)min((int64_t)128, (int64_t)gr.last - S0) : 0;

  // lane (r0, q) loads columns 4q .. and 64 + 4q .. of rows r0 and r0 + 16 of a
  // block, all four in flight; rows behind the group's last are zeros
  const int q = tid & 15, r0 = tid >> 4;
  int from[8];                                         // source rows of all four blocks: their
#pragma unroll                                         // loads then wait for no index
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    from[i] = r < rows ? (int)source_row(a, S0 + r) : -1;
  }
  u32x2 v[4];
  auto load = [&](int s0, int s1) {
    const int64_t c = C0 + 4 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[2 * h] = v[2 * h + 1] = u32x2{0u, 0u};
      const int s = h ? s1 : s0;
      if (s >= 0) {
        const uint16_t *p = a.x + (int64_t)s * a.ld + c;
        if (c < cols) v[2 * h] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
        if (c + 64 < cols)
          v[2 * h + 1] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p + 64));
      }
    }
  };
  load(from[0], from[1]);
  float sum = 0.0f;                                    // of this thread's column (axis 0)
#pragma unroll 1
  for (int block = 0; block < 4; ++block) {
    const int live = rows - 32 * block;                // rows of the block, <= 0: none
    const int64_t R0 = S0 + 32 * block;
    if (block) __syncthreads();                        // the last block is read
    if (live > 0) {
      float *d = st + r0 * kPitch + 4 * q;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4 *>(d + (k >> 1) * 16 * kPitch + (k & 1) * 64) =
            make_float4(bits_f(v[k].x << 16), bits_f(v[k].x & 0xFFFF0000u), bits_f(v[k].y << 16),
                        bits_f(v[k].y & 0xFFFF0000u));
      if (block == 0) load(from[2], from[3]);
      if (block == 1) load(from[4], from[5]);
      if (block == 2) load(from[6], from[7]);
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
      if (r >= end1 || kb >= nsl1 * 4) continue;
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
      } else {                                         // rows of no group, padding of K
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = 0u;
        s = 0u;
      }
      *reinterpret_cast<uint4 *>(a.codes1 + code_offset(r, kb, nsl1)) =
          make_uint4(out[0], out[1], out[2], out[3]);
      a.scales1[scale_offset(r, kb, mnp1)] = (uint8_t)s;
      continue;
    }
    // axis 0: column C0 + cc, block kb along the rows
    const int cc = tid - 128;
    const int64_t c = C0 + cc;                         // < mnp0 (grid)
    const int64_t kb = (int64_t)by * 4 + block;
    uint32_t mask = 0u;
    if (ROT == MX_K_ROT_RAND_SIGN)                     // the index within the group's K
      mask = gather_sign_mask(
          sign_nibble((uint32_t)(((by - gr.before) * 4 + block) * 8 + (lane & 7)), a.seed0_lo), 0);
    if (live > 0 && c < cols) {                        // uniform over each quad (cols % 32 == 0)
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = st[j * kPitch + cc];
      if (a.partial) sum += sum_of<0, 32>(y);          // (rows behind the last are zeros)
      if (!a.codes0) continue;
      if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
      rotate_block<ROT>(y);
      if (RND == MX_K_ROUND_SR) {
        // element (row, c) draws word c % 4 of the call at (row cols + c) / 4;
        // the four lanes of a quad share each call (see quant_axis0_sr_kernel)
        float m1, m2;
        s = block_scale<RotKind<ROT>::value>(y, m1, m2);
        const uint32_t qq = (uint32_t)(cc & 3);
        const uint64_t lq0 = (uint64_t)R0 * (uint64_t)cols + (uint64_t)(c & ~(int64_t)3);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = 0u;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const U4 w = sr_words((lq0 + (uint64_t)(i + (int)qq) * (uint64_t)cols) >> 2, a.seed0_lo,
                                a.seed0_hi);
          const uint32_t own = pick_word(w, qq);
          const uint32_t g1 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, qq ^ 1u),
                                                                    0xB1, 0xF, 0xF, false);
          const uint32_t g2 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, qq ^ 2u),
                                                                    0x4E, 0xF, 0xF, false);
          const uint32_t g3 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)pick_word(w, qq ^ 3u),
                                                                    0x1B, 0xF, 0xF, false);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t d = (uint32_t)r ^ qq;
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
    } else {                                           // K padding of the operand
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = 0u;
      s = 0u;
    }
    if (!a.codes0 || by >= nsl0) continue;
    *reinterpret_cast<uint4 *>(a.codes0 + code_offset(c, kb, nsl0)) =
        make_uint4(out[0], out[1], out[2], out[3]);
    a.scales0[scale_offset(c, kb, mnp0)] = (uint8_t)s;
  }
  if (a.partial && tid >= 128 && in_group && C0 + tid - 128 < cols)
    a.partial[(int64_t)by * cols + C0 + tid - 128] = sum;
}

// The axis-1 operand alone: a wave encodes one tile, 16 rows x 128 K elements, as
// quant_axis1_kernel does. Of the groups it needs only where the last one ends,
// which is looked up while the rows are on their way.
template <int ROT, int RND>
__global__ __launch_bounds__(256, 6) void quant_gather_kernel(GroupedQuantArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t stage[4][4096];
  const int64_t mnp = ((int64_t)a.rows + 255) & ~(int64_t)255;
  const uint32_t nslices = (uint32_t)((a.cols + 127) >> 7);
  const uint32_t ntiles = (uint32_t)(mnp >> 4) * nslices;      // below 2^32: codes < 1 GiB
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t tile = blockIdx.x * 4u + (uint32_t)wv;
  if (tile >= ntiles) return;
  uint8_t *st = stage[wv];
  const uint32_t g = tile / nslices, q = tile - g * nslices;   // (row group, K slice)
  {
    // instruction j reads rows 4j .. 4j + 3, 16 lanes per row; columns past the
    // source are read from its last chunk (only padding blocks use them)
    const int ch = lane & 15;
    const int64_t k = min((int64_t)q * 128 + ch * 8, a.cols - 8);
    u32x4 v[4];
    int64_t s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s[j] = source_row(a, min((int64_t)g * 16 + j * 4 + (lane >> 4), (int64_t)a.rows - 1));
#pragma unroll
    for (int j = 0; j < 4; ++j)                        // (rows of zeros: from row 0)
      v[j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4 *>(a.x + max(s[j], (int64_t)0) * a.ld + k));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rr = j * 4 + (lane >> 4);
      if (s[j] < 0) v[j] = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4 *>(st + rr * 256 + ((ch ^ rr) << 4)) = v[j];
    }
  }
  int last = 0;                                        // behind the last group's last row
  if (a.ends)
    for (int e = lane; e < a.groups; e += 64) last = max(last, a.ends[e]);
  else
    last = a.rows;
  last = __builtin_amdgcn_readlane(scan_max(last), 63);
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

  const int rr = lane & 15, cb = lane >> 4;
  const int64_t r = (int64_t)g * 16 + rr, kb = (int64_t)q * 4 + cb;
  uint32_t mask = 0u;
  if (ROT == MX_K_ROT_RAND_SIGN) {
    // the tile's 128 indices need 32 sign calls: lane l makes call l % 32
    const uint32_t nib = sign_nibble(q * 32 + (lane & 31), a.seed1_lo);
    const uint32_t m0 = gather_sign_mask(nib, 0), m1 = gather_sign_mask(nib, 8),
                   m2 = gather_sign_mask(nib, 16), m3 = gather_sign_mask(nib, 24);
    mask = cb == 0 ? m0 : cb == 1 ? m1 : cb == 2 ? m2 : m3;
  }
  float y[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4 d = *reinterpret_cast<const u32x4 *>(st + rr * 256 + (((cb * 4 + j) ^ rr) << 4));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      y[8 * j + 2 * t] = bits_f(d[t] << 16);
      y[8 * j + 2 * t + 1] = bits_f(d[t] & 0xFFFF0000u);
    }
  }
  if (ROT == MX_K_ROT_RAND_SIGN) apply_sign_mask(y, mask);
  rotate_block<ROT>(y);
  const uint64_t q0 = (uint64_t)(r * a.cols + (kb << 5)) >> 2;
  U4 w{0u, 0u, 0u, 0u};
  auto u24_of = [&](int i) -> uint32_t {
    if ((i & 3) == 0) w = sr_words(q0 + (uint64_t)(i >> 2), a.seed1_lo, a.seed1_hi);
    return pick_word(w, (uint32_t)(i & 3)) >> 8;
  };
  uint32_t out[4];
  uint32_t s = quantize_block<RotKind<ROT>::value, RND, kFmtE2M1>(y, out, u24_of);
  if (r >= min(last, a.rows) || (kb << 5) >= a.cols) { // rows of no group, padding
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 0u;
    s = 0u;
  }
  *reinterpret_cast<uint4 *>(a.codes1 + (size_t)tile * 1024 + lane * 16) =
      make_uint4(out[0], out[1], out[2], out[3]);
  a.scales1[scale_offset(r, kb, mnp)] = (uint8_t)s;
}

// sums[e][c] = the partial sums of group e's slices. A workgroup has 64 columns
// and four waves that take every fourth slice each; their sums meet in LDS.
__global__ __launch_bounds__(256) void group_sums_kernel(GroupedQuantArgs a, uint32_t gx) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (int)(blockIdx.x / gx);
  const int64_t c = (int64_t)(blockIdx.x % gx) * 64 + lane;
  const Group gr = find_group<false>(a.ends, a.groups, a.rows, a.each, e, CountSlices());
  const int slices = CountSlices()(gr.first, gr.last);
  float sum = 0.0f;
  if (c < a.cols) {
    const float *p = a.partial + (int64_t)gr.before * a.cols + c;
#pragma unroll 4
    for (int b = wave; b < slices; b += 4) sum += p[(int64_t)b * a.cols];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && c < a.cols)
    a.sums[(int64_t)e * a.cols + c] =
        (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

template <int ROT, int RND>
hipError_t launch_grouped(const GroupedQuantArgs &a, hipStream_t stream) {
  if (!a.codes0 && !a.sums) {
    const int64_t tiles = (((int64_t)a.rows + 255) / 256 * 16) * ((a.cols + 127) / 128);
    return launch(quant_gather_kernel<ROT, RND>, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0,
                  stream, a);
  }
  const int64_t gx = ((a.cols + 255) & ~(int64_t)255) / 128;
  // the groups' slices, and behind them whichever is longer of the slices left
  // and the axis-1 operand's rows in no group: 4 slices more hold the latter
  const int64_t gy = (int64_t)a.slices + 4;
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
