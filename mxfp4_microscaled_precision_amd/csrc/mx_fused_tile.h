// Products with an epilogue and products grouped by expert, in tiles of 256
// columns and 256 or 128 rows: MXFP4 operands in the packed tile layout (see
// mxfp4.h), fp32 sums.
//
// The pipeline is that of the plain product (mx_gemm.hip): one persistent
// workgroup per compute unit, eight waves that multiply and four that only copy
// 128-deep stages into a ring of four LDS buffers, direct-to-LDS, three stages
// ahead and across tiles. What differs:
//
//  * Tiles belong to groups of rows whose ends only the device knows. Each
//    workgroup makes a table of the groups in LDS when it starts, so a tile's
//    group is a look-up without memory, and copies in flight are never waited
//    for on its account.
//  * A tile begins at a multiple of 64 rows of the operand (the scales of 64
//    rows are 256 contiguous bytes, copied quarter by quarter), wherever its
//    group begins; rows of other groups are neither copied nor multiplied
//    where a whole 16-row tile of them lies outside, nor stored.
//  * A tile with at most 128 rows left is 128 rows high: both wave rows then
//    have half of it. The last round of tiles is cut in halves as well if they
//    would fill at most half of the compute units.
//  * K is a tile's own: a slice range of either operand, which may be empty.
//  * The epilogue (mx_epilogue.h) works on the registers that hold the sums, 16
//    bytes a lane and access (at any alignment), or by columns through LDS in the
//    64 columns where the matrix ends, and where its rows are 16 MB or more apart.
//
// Bound by two things one after the other: the stages by the matrix instructions
// (8192x14336x4096 alone: 201 us, 4.8 PFLOP/s, what the card's power allows), the
// epilogue by memory (the gate's mul, pre and C are 705 MB, 137 us at a copy's
// rate); measured 343 to 358 us together, call after call, in which 649 MB are read
// and 473 written, 3.2 of the 5.16 TB/s that a copy reaches. While a wave's 128 sums
// a lane wait for their epilogue no register is left for another tile's. Starting
// half of the workgroups later, so that some multiply while others store, changed
// nothing; no counter was taken that says why.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "mx_epilogue.h"
#include "mx_gemm_common.h"
#include "mx_groups.h"
#include "mx_kernels.h"

namespace mx {

namespace tile {

using namespace gemm;

constexpr int kThreads = 768;                      // 8 multiplying + 4 copying waves
constexpr int kConsumers = 8;
constexpr int kStageA = kBM * 64;                  // 16 tiles of 1 KB
constexpr int kStageB = kBN * 64;
constexpr int kStageSA = kBM * 4;                  // four 256-byte quarters of scales
constexpr int kStageSB = kBN * 4;
constexpr int kStageBytes = kStageA + kStageB + kStageSA + kStageSB;
constexpr int kRing = 4;
constexpr int kAhead = kRing - 1;
constexpr int kRows = 8;                           // 16-row strips of a wave's part, at most
constexpr int kColumns = kRing * kStageBytes + kConsumers * kSlab;   // bias of each wave's 64
constexpr int kTable = kColumns + kConsumers * 64 * 4;
// groups that the table has room for (two words each)
constexpr int kTileGroups = (160 * 1024 - kTable) / 8;
static_assert(kTileGroups >= 768, "LDS");

// The launch's tiles, the same for every workgroup.
struct Plan {
  int row_tiles, col_tiles;        // of all groups
  int total, whole;                // tiles; those that are not cut in halves
  int mine;                        // tiles (or halves) of this workgroup
};

// One tile: rows ra .. ra + h - 1 of A (C rows c_row + them, those in [first,
// last)), rows rb .. rb + 255 of B (C columns col0 ..), nk slices from ka, kb.
struct Tile {
  int e, ra, h, first, last, rb, col0, ka, kb, nk;
  bool live;                       // has any slice
};

// The kernel's arguments, from memory: held in scalar registers through the stage
// loop they would spill (the compiler cannot tell that it read them before).
__device__ __forceinline__ const FusedArgs &read_again() {
  auto args = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(args));
  return *(const FusedArgs *)args;
}

// Table of the groups in LDS: where each ends, and the tiles (or, for weight
// gradients, slices) up to and with it. One wave fills it.
__device__ __forceinline__ void fill_table(const FusedArgs &g, int *ends, int *units) {
  const int lane = (int)__lane_id();
  int row = 0, before = 0;
  for (int base = 0; base < g.groups; base += 64) {
    const int e = base + lane;
    int last = e < g.groups ? min(max(g.ends[e], 0), g.rows) : 0;
    last = max(scan_max(last), row);
    const int first = __builtin_amdgcn_update_dpp(row, last, 0x138, 0xF, 0xF, false);
    int n = 0;
    if (e < g.groups)
      n = g.kind == MX_K_WGRAD ? CountSlices()(first, last) : CountTiles<kBM, 64>()(first, last);
    n = scan_add(n) + before;
    if (e < g.groups) {
      ends[e] = last;
      units[e] = n;
    }
    row = __builtin_amdgcn_readlane(last, 63);
    before = __builtin_amdgcn_readlane(n, 63);
  }
}

__device__ __forceinline__ int uniform_word(const int *p) {
  return __builtin_amdgcn_readfirstlane(*p);
}

// Group of row tile rt: the first whose tiles go past it.
__device__ __forceinline__ int group_of(const int *units, int groups, int rt) {
  const int lane = (int)__lane_id();
  for (int base = 0; base < groups; base += 64) {
    const int e = base + lane;
    const uint64_t past = __ballot(e < groups && units[e < groups ? e : 0] > rt);
    if (past) return base + __builtin_ctzll(past);
  }
  return groups - 1;               // rt is below the last group's (see Plan)
}

__device__ __forceinline__ Plan make_plan(const FusedArgs &g, const int *units) {
  Plan p;
  const int bid = (int)blockIdx.x, grid = (int)gridDim.x;
  const int tm = (g.M + kBM - 1) / kBM;
  p.row_tiles = g.kind == MX_K_WGRAD ? g.groups * tm
                : g.ends             ? uniform_word(units + g.groups - 1)
                                     : tm;
  p.col_tiles = g.col_tiles;
  p.total = p.row_tiles * p.col_tiles;
  const int rem = p.total % grid;
  const bool cut = rem != 0 && 2 * rem <= grid;
  p.whole = cut ? p.total - rem : p.total;
  p.mine = bid < p.whole ? (p.whole - bid + grid - 1) / grid : 0;
  if (cut && bid < 2 * rem) ++p.mine;
  return p;
}

// This workgroup's k-th tile.
__device__ __forceinline__ Tile tile_at(const FusedArgs &g, const Plan &p, const int *ends,
                                        const int *units, int k) {
  const int bid = (int)blockIdx.x, grid = (int)gridDim.x;
  // Workgroups go round-robin over the 8 XCDs. Every round of tiles is a consecutive
  // run of them, and each XCD's share of it is as well, in groups of kGroupM tile
  // rows (see tile_coords). With a run of all rounds' tiles for each XCD instead,
  // the XCDs read and wrote eight far places of the matrices at a time (8192x8192x2048,
  // us: bf16 with mul and pre 188, now 152; fp32 with mul and residual 234, now 200;
  // gradient with dmul 196, now 162), and one XCD had the weight gradient of the
  // experts with the most rows (8 experts, 16384 rows, 4096x4096: 413 to 442, now 317).
  int id = bid + k * grid, half = -1;
  if (id < p.whole) {
    const int base = id - bid, n = min(grid, p.whole - base);
    const int x = bid & 7, each = n >> 3, more = n & 7;
    id = base + x * each + min(x, more) + (bid >> 3);
  } else {
    id = p.whole + (bid >> 1);
    half = bid & 1;
    if (p.whole == p.total) half = -1;      // (not reached: mine counts no such tile)
  }
  static_assert(kGroupM == 4, "divisions below");
  const int grp = g.by_col_tiles(id >> 2), first_row = grp * kGroupM;
  const int gm = min(kGroupM, p.row_tiles - first_row);
  const int r = id - grp * kGroupM * p.col_tiles;
  const int ct = gm == 4 ? r >> 2 : gm == 3 ? r / 3 : gm == 2 ? r >> 1 : r;
  const int rt = first_row + r - ct * gm;

  Tile t;
  t.e = 0;
  t.first = 0;
  t.last = g.M;
  t.ka = t.kb = 0;
  t.nk = g.a_slices;
  t.rb = t.col0 = ct * kBN;
  if (g.kind == MX_K_WGRAD) {
    const int tm = (g.M + kBM - 1) / kBM;
    t.e = g.by_row_tiles(rt);
    t.ra = (rt - t.e * tm) * kBM;
    t.ka = t.kb = t.e ? uniform_word(units + t.e - 1) : 0;
    t.nk = uniform_word(units + t.e) - t.ka;
  } else if (!g.ends) {
    t.ra = rt * kBM;
  } else {
    t.e = group_of(units, g.groups, rt);
    t.first = t.e ? uniform_word(ends + t.e - 1) : 0;
    t.last = uniform_word(ends + t.e);
    t.ra = (t.first & ~63) + (rt - (t.e ? uniform_word(units + t.e - 1) : 0)) * kBM;
    if (g.kind == MX_K_DGRAD) {
      t.kb = t.e * g.a_slices;
    } else {
      const int at = t.e * g.N;             // the group's first row of B (< 2^24)
      t.rb = (at & ~63) + ct * kBN;
      t.col0 = t.rb - at;
    }
  }
  t.h = kBM;
  if (half >= 0) {
    t.h = kBM / 2;
    t.ra += half * (kBM / 2);
  } else if (t.last - t.ra <= kBM / 2) {
    t.h = kBM / 2;
  }
  t.live = t.nk > 0;
  t.nk = max(t.nk, 1);                      // an empty sum: one stage of zeros
  return t;
}

// The 4 MFMAs of strip I.
template <int I>
__device__ __forceinline__ void multiply_strip(v4f (&acc)[kRows][4], const uint4 (&bf)[4],
                                               const uint4 &af, uint32_t sb, uint2 sa) {
  const uint32_t sai = I < 4 ? sa.x : sa.y;
  acc[I][0] = mfma_fp4<0, I & 3>(bf[0], af, acc[I][0], sb, sai);
  acc[I][1] = mfma_fp4<1, I & 3>(bf[1], af, acc[I][1], sb, sai);
  acc[I][2] = mfma_fp4<2, I & 3>(bf[2], af, acc[I][2], sb, sai);
  acc[I][3] = mfma_fp4<3, I & 3>(bf[3], af, acc[I][3], sb, sai);
}

// Strip I of the LIVE that a wave's stage has: read the A fragment two strips on
// (in strip S - 1 every one still unread), then multiply. See consume_row in
// mx_gemm.hip.
template <int I, int S, int LIVE>
__device__ __forceinline__ void strip(v4f (&acc)[kRows][4], const uint4 (&bf)[4],
                                      uint4 (&af)[LIVE], const uint8_t *a_base, uint32_t sb,
                                      uint2 sa) {
  if (I < S) {
#pragma unroll
    for (int j = I + 2; j < (I == S - 1 ? LIVE : I + 3); ++j)
      if (j < LIVE) af[j < LIVE ? j : 0] = *reinterpret_cast<const uint4 *>(a_base + j * 1024);
  }
  multiply_strip<I>(acc, bf, af[I], sb, sa);
  __builtin_amdgcn_sched_barrier(0);
}

template <int LO, int S, int LIVE, int... I>
__device__ __forceinline__ void strips(std::integer_sequence<int, I...>, v4f (&acc)[kRows][4],
                                       const uint4 (&bf)[4], uint4 (&af)[LIVE],
                                       const uint8_t *a_base, uint32_t sb, uint2 sa) {
  (strip<LO + I, S, LIVE>(acc, bf, af, a_base, sb, sa), ...);
}

// Strips 0 .. live - 1 of a stage, any number: each read when it is multiplied.
template <int... I>
__device__ __forceinline__ void some_strips(std::integer_sequence<int, I...>, v4f (&acc)[kRows][4],
                                            const uint4 (&bf)[4], const uint8_t *a_base,
                                            uint32_t sb, uint2 sa, int live) {
  auto one = [&](auto i) {
    if (i() < live) {
      const uint4 af = *reinterpret_cast<const uint4 *>(a_base + i() * 1024);
      multiply_strip<i()>(acc, bf, af, sb, sa);
    }
  };
  (one(std::integral_constant<int, I>()), ...);
}

// Eight rows (half s of strip s / 2) of the wave's sums into its 2 KB of LDS:
// lane (lr, lg) holds columns 16 j + 4 lg .. + 3 of row lr of a strip and
// writes them as 16-byte chunk 4 j + lg of the row, at chunk ^ 2 (row % 8): a
// row's 256 bytes are all 64 banks, without it the eight rows would collide.
// One body for all steps: only the accumulators are named in it (unrolled
// sixteen times the epilogue would be some 100 KB of code).
__device__ __forceinline__ void stage_rows(const v4f (&acc)[kRows][4], uint8_t *slab, int s, int lane) {
  const int lr = lane & 15, lg = lane >> 4;
  if ((lr >> 3) == (s & 1)) {
    uint8_t *to = slab + (lr & 7) * 256;
    const int swap = 2 * (lr & 7);
#define MX_STRIP(I)                                                               \
  case I:                                                                         \
    _Pragma("unroll") for (int j = 0; j < 4; ++j)                                 \
        *reinterpret_cast<v4f *>(to + (((4 * j + lg) ^ swap) << 4)) = acc[I][j];  \
    asm volatile("; strip %0" ::"i"(I) : "memory"); /* else one store, acc indexed */ \
    break;
    switch (s >> 1) {
      MX_STRIP(0) MX_STRIP(1) MX_STRIP(2) MX_STRIP(3)
      MX_STRIP(4) MX_STRIP(5) MX_STRIP(6) MX_STRIP(7)
    }
#undef MX_STRIP
  }
}

// The wave's LDS accesses stay in program order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// f(0), f(1), .. f(N - 1) with the numbers as constants.
template <typename F, int... I>
__device__ __forceinline__ void for_ints(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each_int(F f) {
  for_ints(f, std::make_integer_sequence<int, N>());
}

// A matrix of the epilogue from the wave's first row and column on, as a buffer:
// accesses at kOutside or beyond do nothing.
constexpr uint32_t kOutside = 0x80000000u;
struct Rows {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t pitch;                                  // bytes; 128 rows stay below kOutside (host)
  bool any;
  __device__ __forceinline__ Rows(const void *base, int64_t ld, int64_t row, int64_t col, int esize)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(
            base ? static_cast<uint8_t *>(const_cast<void *>(base)) + (row * ld + col) * esize
                 : nullptr,
            0, base ? kOutside : 0, 0x00020000)),
        pitch((uint32_t)(ld * esize)), any(base != nullptr) {}
  // `byte` bytes past the lane's offset in row `row` (both uniform)
  __device__ __forceinline__ row_u32x4 load(uint32_t at, uint32_t row, uint32_t byte) const {
    return __builtin_bit_cast(
        row_u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, row * pitch + byte, 0));
  }
  // With the row's offset in the lanes' own, not in the instruction's scalar
  // register: behind a store with a scalar offset the compiler lets the very next
  // instruction write the registers that are being stored, and the store has been
  // seen to write that instruction's result now and then (one 16-byte unit's first
  // word). Without one it keeps the two instructions' distance that the store needs.
  __device__ __forceinline__ void store(row_u32x4 v, uint32_t at, uint32_t row,
                                        uint32_t byte) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, at + (row * pitch + byte), 0, 0);
  }
};

// Lanes 8 .. 15 of each 16 in `a` and lanes 0 .. 7 of each in `b` change places.
__device__ __forceinline__ void swap_halves(float &a, float &b) {
  const int x = (int)f_bits(a), y = (int)f_bits(b);
  a = bits_f((uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false));
  b = bits_f((uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false));
}

// The wave's part of a finished tile, 16-byte accesses, from the registers that
// hold it: no LDS, no waits between the waves.
//
// Lane (lr, lg) holds columns 16 j + 4 lg .. + 3 of row lr of each strip, j < 4,
// for fp32 a unit of 16 bytes. For bf16 the odd and even 16-lane rows of two
// neighbouring j are swapped, after which the lane has eight adjacent columns,
// 32 p + 16 (lg % 2) + 8 (lg / 2) .. of pair p: eight instructions a strip, where
// staging rows of 64 columns in LDS took some 260 and most of the epilogue's time.
// An access is then 64 bytes of 16 rows. With LINES the upper eight rows of one
// unit and the lower eight of the next change places first, 24 instructions a
// strip, and it is 128 bytes, a line, of eight rows: worth it where three or four
// matrices are read and written (8192x8192x2048, us without and with: fp32 with
// mul and residual 268 -> 234, with mul and pre 306 -> 274; gradients with dmul
// fp32 328 -> 310, bf16 206 -> 196), and not elsewhere (gradients alone fp32
// 197 -> 199, bf16 122 -> 124; experts' bf16 rows with mul 205 -> 213).
//
// mul, the residual or pre of a unit are asked for one unit ahead at first, and
// further once the accumulators of finished units leave registers for them; each
// request goes out before its unit's stores, so that no load waits for a store.
template <int F32, int MODE, int ACT>
__device__ __forceinline__ void finish_rows(const FusedArgs &g, const Tile &t,
                                            v4f (&acc)[kRows][4], const float *columns,
                                            int64_t c_row, int row0, int col0, int live, int lane) {
  constexpr bool GRAD = is_gradient(MODE);
  constexpr int kSize = F32 ? 4 : 2, n = kUnit<F32>;
  constexpr int kPerStrip = F32 ? 4 : 2;           // units of a lane in a strip
  constexpr int kUnits = kPerStrip * kRows;
  // two matrices to read, or one (which a forward call chooses)
  constexpr bool TWO = MODE == kForwardBoth || MODE == kGradientMul;
  constexpr bool LINES = F32 ? MODE != kGradient : MODE == kGradientMul;
  const bool gate = !GRAD && g.e.mul;
  const Rows pm(TWO ? g.e.mul : nullptr, g.e.ldmul, c_row + row0, col0, kSize);
  const Rows po(!TWO && gate ? g.e.mul : other_of<GRAD>(g.e),
                !TWO && gate ? g.e.ldmul : other_ld<GRAD>(g.e), c_row + row0, col0, kSize);
  const Rows p2(second_of<GRAD>(g.e), second_ld<GRAD>(g.e), c_row + row0, col0, kSize);
  const Rows pc(g.c, g.ldc, c_row + row0, col0, kSize);
  // Byte of this lane in a strip of matrix m: one multiply-add, made anew at every
  // use (the compiler would hold one register per matrix, and spill). Rows that
  // are not the tile's are outside.
  const int lg = lane >> 4;
  const uint32_t lr = lane & (LINES ? 7 : 15), side = LINES ? lane >> 3 & 1 : 0;
  const uint32_t c0 = (F32 ? 16 * side + 4 * lg : 32 * side + 16 * (lg & 1) + 8 * (lg >> 1)) * kSize;
  // a unit's first row in the part, and its first byte in the row
  constexpr auto row_of = [](int u) { return u / kPerStrip * 16 + (LINES ? 8 * (u & 1) : 0); };
  constexpr auto byte_of = [](int u) {
    return LINES ? (u % kPerStrip >> 1) * 128 : u % kPerStrip * 64;
  };
  const int before = t.first - row0, count = t.last - t.first;
  auto at = [&](const Rows &m, int row) {
    uint32_t b;
    asm volatile("v_mad_u32_u24 %0, %1, %2, %3" : "=v"(b) : "v"(lr), "s"(m.pitch), "v"(c0));
    return lr + (uint32_t)(row - before) < (uint32_t)count ? b : kOutside;
  };
  // the last unit asked for when unit u is done: kMost units ahead at most
  constexpr int kMost = TWO ? 4 : 10, kSlots = kMost + 1;
  constexpr int kWait = GRAD ? 2 * kPerStrip : kPerStrip;
  constexpr int kSlow = (F32 ? 2 : 1) * (TWO ? GRAD ? 3 : 2 : 1);
  constexpr auto requested = [](int u) {
    const int more = u < kWait ? 0 : (u - kWait) / kSlow;
    return u + 1 + (more < kMost - 1 ? more : kMost - 1);
  };
  row_u32x4 mul[TWO ? kSlots : 1], other[kSlots];
  auto load = [&](auto unit) {
    constexpr int u = unit();
    constexpr int i = u / kPerStrip, row = row_of(u), byte = byte_of(u);
    if (u >= kUnits || i >= live) return;
    if constexpr (TWO) mul[u % kSlots] = pm.load(at(pm, row), row, byte);
    if (TWO || GRAD || po.any) other[u % kSlots] = po.load(at(po, row), row, byte);
  };
  load(std::integral_constant<int, 0>());
  for_each_int<kUnits>([&](auto unit) {
    constexpr int u = unit(), i = u / kPerStrip, q = u % kPerStrip;
    constexpr int row = row_of(u), byte = byte_of(u);
    if (i < live) {
      if constexpr (LINES && q % 2 == 0) {
#pragma unroll
        for (int j = 0; j < (F32 ? 1 : 2); ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float a = acc[i][q + j][k], b = acc[i][q + j + (F32 ? 1 : 2)][k];
            swap_halves(a, b);
            acc[i][q + j][k] = a;
            acc[i][q + j + (F32 ? 1 : 2)][k] = b;
          }
      }
      float v[n];
      if constexpr (F32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = acc[i][q][k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const auto r = __builtin_amdgcn_permlane16_swap(
              f_bits(acc[i][2 * q][k]), f_bits(acc[i][2 * q + 1][k]), false, false);
          v[k] = bits_f(r[0]);
          v[k + 4] = bits_f(r[1]);
        }
      }
      if (!GRAD && g.e.bias) {
#pragma unroll
        for (int k = 0; k < n; k += 4) {
          const v4f b = *reinterpret_cast<const v4f *>(columns + (c0 + byte) / kSize + k);
#pragma unroll
          for (int h = 0; h < 4; ++h) v[k + h] += b[h];
        }
      }
      row_u32x4 c, second;
      epilogue_unit<F32, MODE, ACT>(v, TWO || gate, TWO || (po.any && !gate),
                                    TWO ? mul[TWO ? u % kSlots : 0] : other[u % kSlots],
                                    other[u % kSlots], c, second);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int done = u == 0 ? 0 : requested(u - 1), more = requested(u) - done;
      load(std::integral_constant<int, done + 1>());
      if constexpr (more > 1) load(std::integral_constant<int, done + 2>());
      // (a store into no matrix does nothing; a branch around it would move what
      // it stores behind it, and hold every element's exponential up to there)
      if (GRAD ? MODE == kGradientMul : p2.any) p2.store(second, at(p2, row), row, byte);
      pc.store(c, at(pc, row), row, byte);
      __builtin_amdgcn_sched_barrier(0);
    }
  });
}

// The same element by element, where 64 columns are not all the matrix's:
// the sums go through LDS, eight rows at a time, and lane l has column l of four
// rows at once, so that 64 lanes still access 64 adjacent columns.
template <int F32, int MODE, int ACT>
__device__ __forceinline__ void finish_columns(const FusedArgs &g, const Tile &t,
                                               const v4f (&acc)[kRows][4], uint8_t *slab,
                                               const float *columns, int64_t c_row, int row0,
                                               int col0, int live, int lane) {
  constexpr bool GRAD = is_gradient(MODE);
#pragma clang loop unroll(disable)
  for (int s = 0; s < 4 * live; ++s) {             // four rows, half s % 2 of eight
    int l = lane;
    asm volatile("" : "+v"(l));
    const int col = col0 + l, r0 = row0 + 4 * s;
    const bool in = col >= 0 && col < g.N;
    if (!(s & 1)) {
      wave_sync();
      stage_rows(acc, slab, s >> 1, l);
      wave_sync();
    }
    const void *const from = other_of<GRAD>(g.e);
    float v[4], m[4], o[4], a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + i, at = 4 * (s & 1) + i;
      const bool mine = in && row >= t.first && row < t.last;
      m[i] = o[i] = 0.0f;
      if (mine && g.e.mul) m[i] = load_one<F32>(g.e.mul, (c_row + row) * g.e.ldmul + col);
      if (mine && from) o[i] = load_one<F32>(from, (c_row + row) * other_ld<GRAD>(g.e) + col);
      v[i] = *reinterpret_cast<const float *>(slab + at * 256 + (((l >> 2) ^ (2 * at)) << 4) +
                                              (l & 3) * 4);
      if (!GRAD && g.e.bias) v[i] += columns[l];
    }
    epilogue_of<MODE, ACT>(
        v, [&](int k) { return m[k]; }, [&](int k) { return o[k]; }, g.e.mul, g.e.residual, a, b);
    void *const to2 = second_of<GRAD>(g.e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + i;
      if (!in || row < t.first || row >= t.last) continue;
      if (to2) store_one<F32>(to2, (c_row + row) * second_ld<GRAD>(g.e) + col, b[i]);
      store_one<F32>(g.c, (c_row + row) * g.ldc + col, a[i]);
    }
  }
}

// The wave's part of a finished tile: `live` strips of 16 rows x 64 columns. The
// bias of its columns waits in LDS (`columns`): eight registers less.
template <int F32, int MODE, int ACT>
__device__ __forceinline__ void finish(const Tile &t, v4f (&acc)[kRows][4], uint8_t *slab, float *columns,
                                       int row0, int col0, int live, int lane) {
  const FusedArgs &g = read_again();
  if (live == 0 || col0 >= g.N || col0 + 64 <= 0) return;
  asm volatile("" : "+v"(lane));                   // keeps lane addresses out of the stage loop
  const int64_t c_row = g.kind == MX_K_WGRAD ? (int64_t)t.e * g.M : 0;
  const int col = col0 + lane;
  columns[lane] =
      g.e.bias && col >= 0 && col < g.N ? load_bias(g.e, (int64_t)t.e * g.N + col) : 0.0f;
  wave_sync();
  const bool vec = g.e.vec && col0 >= 0 && col0 + 64 <= g.N;
  if (vec)
    finish_rows<F32, MODE, ACT>(g, t, acc, columns, c_row, row0, col0, live, lane);
  else
    finish_columns<F32, MODE, ACT>(g, t, acc, slab, columns, c_row, row0, col0, live, lane);
}

// One tile's stages, from stage G of the ring on, of LIVE strips (0: of `live`).
// SHIFTED waves run most of a stage behind, and take the barrier where they have
// read all of it (see consumer_loop in mx_gemm.hip).
template <bool SHIFTED, int LIVE>
__device__ __forceinline__ void stages(v4f (&acc)[kRows][4], const uint8_t *smem, int G, int nk,
                                       uint32_t a_off, uint32_t b_off, uint32_t sa_off,
                                       uint32_t sb_off, int live) {
  constexpr int kSplit = LIVE == kRows ? 6 : 3;
  for (const int end = G + nk; G < end; ++G) {
    if (!SHIFTED) __syncthreads();                         // stage G landed
    const uint8_t *base = smem + (G & 3) * kStageBytes;
    uint4 bf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const uint4 *>(base + b_off + j * 1024);
    const uint32_t sb = *reinterpret_cast<const uint32_t *>(base + sb_off);
    // (four strips or fewer: the second word is other rows', unused)
    const uint2 sa = make_uint2(*reinterpret_cast<const uint32_t *>(base + sa_off),
                                *reinterpret_cast<const uint32_t *>(base + sa_off + 256));
    if constexpr (LIVE == 0) {
      some_strips(std::make_integer_sequence<int, kRows>{}, acc, bf, base + a_off, sb, sa, live);
      if (SHIFTED) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __syncthreads();
      }
    } else {
      uint4 af[LIVE];
      af[0] = *reinterpret_cast<const uint4 *>(base + a_off);
      af[1] = *reinterpret_cast<const uint4 *>(base + a_off + 1024);
      if (!SHIFTED) {
        strips<0, LIVE, LIVE>(std::make_integer_sequence<int, LIVE>{}, acc, bf, af, base + a_off,
                              sb, sa);
      } else {
        strips<0, kSplit, LIVE>(std::make_integer_sequence<int, kSplit>{}, acc, bf, af,
                                base + a_off, sb, sa);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); // all of stage G read
        __syncthreads();                                   // stage G + 1 landed
        strips<kSplit, kSplit, LIVE>(std::make_integer_sequence<int, LIVE - kSplit>{}, acc, bf, af,
                                     base + a_off, sb, sa);
      }
    }
  }
}

// A multiplying wave's tiles; wave row 1 is the shifted one. The two differ in
// their stages only: one copy of the epilogue, which is some 10 KB of code that
// the first tile has to fetch.
template <int F32, int MODE, int ACT>
__device__ __forceinline__ void consume(const Plan &p, uint8_t *smem,
                                        const int *ends, const int *units, int lane, int wm, int wn) {
  uint8_t *slab = smem + kRing * kStageBytes + (wm * 4 + wn) * kSlab;
  float *columns = reinterpret_cast<float *>(smem + kColumns) + (wm * 4 + wn) * 64;
  const uint32_t b_off = (uint32_t)(kStageA + (wn * 4) * 1024 + lane * 16);
  const uint32_t sb_off = (uint32_t)(kStageA + kStageB + kStageSA) + wn * 256 + lane * 4;
  v4f acc[kRows][4];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (wm) __syncthreads();                                 // stage 0 landed
  int G = 0;
  for (int k = 0; k < p.mine; ++k) {
    int live, part;
    {
      const Tile t = tile_at(read_again(), p, ends, units, k);
      part = t.h >> 1;                                     // rows of a wave row: 128 or 64
      live = min(part >> 4, max(0, (t.last - (t.ra + wm * part) + 15) >> 4));
      live = __builtin_amdgcn_readfirstlane(live);
      part = __builtin_amdgcn_readfirstlane(part);
      const int nk = __builtin_amdgcn_readfirstlane(t.nk);
      const uint32_t a_off = (uint32_t)(wm * part * 64 + lane * 16);
      const uint32_t sa_off = (uint32_t)(kStageA + kStageB) + wm * part * 4 + lane * 4;
      if (live == kRows) {
        if (wm)
          stages<true, kRows>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
        else
          stages<false, kRows>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
      } else if (live == kRows / 2) {
        if (wm)
          stages<true, kRows / 2>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
        else
          stages<false, kRows / 2>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
      } else {
        if (wm)
          stages<true, 0>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
        else
          stages<false, 0>(acc, smem, G, nk, a_off, b_off, sa_off, sb_off, live);
      }
      G += nk;
    }
    // the tile is looked up again: what it says would hold registers through
    // the stages
    const Tile t = tile_at(read_again(), p, ends, units, k);
    finish<F32, MODE, ACT>(t, acc, slab, columns, t.ra + wm * part, t.col0 + wn * 64, live, lane);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  if (!wm) __syncthreads();                                // the shifted waves' last barrier
}

template <int F32, int MODE, int ACT>
__global__ __launch_bounds__(kThreads, 1) void fused_tile_kernel(FusedArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kTable];
  __shared__ int ends[kTileGroups], units[kTileGroups];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // 0..11
  if (g.ends) {
    if (wave == kConsumers) fill_table(g, ends, units);
    __syncthreads();
  }
  const Plan plan = make_plan(g, units);
  if (wave < kConsumers) {
    consume<F32, MODE, ACT>(plan, smem, ends, units, lane, wave >> 2, wave & 3);
    return;
  }

  // Copying wave w: row groups 4 w .. 4 w + 3 of A and of B (1 KB tiles); wave
  // 0 the scales of A's 64-row quarters, wave 1 those of B's. Copies of rows
  // outside the tile and stages past the last one read zeros, so that the
  // counts stay the same.
  const int w = wave - kConsumers;
  const uint32_t smem_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);
  const int a_bytes = g.a_panels * g.a_slices * 16384, b_bytes = g.b_panels * g.b_slices * 16384;
  const v4i rsrc_a = make_rsrc(g.a_codes, (uint32_t)a_bytes);
  const v4i rsrc_b = make_rsrc(g.b_codes, (uint32_t)b_bytes);
  const int s_panels = w == 0 ? g.a_panels : g.b_panels;
  const int s_bytes = (w == 0 ? a_bytes : b_bytes) >> 4;
  const v4i rsrc_s = w == 0 ? make_rsrc(g.a_scales, (uint32_t)s_bytes)
                            : make_rsrc(g.b_scales, (uint32_t)s_bytes);
  int ik = 0, is = 0, nk = 0;                              // next stage to copy
  int at_a = 0, at_b = 0, at_s = 0;                        // this lane's first bytes in it
  int live_a = 0;                                          // bit j: row group 4 w + j is the tile's
  bool live_s = false, live = false;
  auto set_tile = [&]() {
    live = ik < plan.mine;
    nk = 1;
    live_a = 0;
    live_s = false;
    if (!live) return;
    const Tile t = tile_at(read_again(), plan, ends, units, ik);
    nk = t.nk;
    live = t.live;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int lo = t.ra + 64 * w + 16 * j;
      if (live && 64 * w + 16 * j < t.h && lo < t.last && lo + 16 > t.first) live_a |= 1 << j;
    }
    at_a = ((t.ra >> 4) + 4 * w) * g.a_slices * 1024 + t.ka * 1024 + lane * 16;
    at_b = ((t.rb >> 4) + 4 * w) * g.b_slices * 1024 + t.kb * 1024 + lane * 16;
    const int q = ((w == 0 ? t.ra : t.rb) >> 6) + (lane >> 4);   // this lane's 64-row quarter
    live_s = live && (q >> 2) < s_panels;
    at_s = ((w == 0 ? t.ka : t.kb) * s_panels + (q >> 2)) * 1024 + (q & 3) * 256 + (lane & 15) * 16;
  };
  set_tile();
  auto issue = [&](int buf) {
    const uint32_t stage = smem_base + (uint32_t)(buf * kStageBytes);
    int al = at_a, bl = at_b, sl = at_s;
    asm volatile("" : "+v"(al), "+v"(bl), "+v"(sl));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t dst = __builtin_amdgcn_readfirstlane(stage + (uint32_t)((w * 4 + j) * 1024));
      dma_load16(rsrc_a, (live_a >> j) & 1 ? al + (j * g.a_slices + is) * 1024 : a_bytes, dst);
      dma_load16(rsrc_b, live ? bl + (j * g.b_slices + is) * 1024 : b_bytes, dst + kStageA);
    }
    if (w < 2)
      dma_load16(rsrc_s, live_s ? sl + is * s_panels * 1024 : s_bytes,
                 __builtin_amdgcn_readfirstlane(
                     stage + (uint32_t)(kStageA + kStageB + (w == 0 ? 0 : kStageSA))));
    if (++is == nk) {
      is = 0;
      ++ik;
      set_tile();
    }
  };
  for (int G = 0; G < kAhead; ++G) issue(G);
  int G = 0;
  for (int k = 0; k < plan.mine; ++k) {
    const int n = tile_at(read_again(), plan, ends, units, k).nk;
    for (int s = 0; s < n; ++s, ++G) {
      // own part of stage G landed, two later stages outstanding
      if (w < 2)
        asm volatile("s_waitcnt vmcnt(18)" ::: "memory");
      else
        asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
      __syncthreads();                                     // stage G visible; G - 1 free
      issue((G + kAhead) & 3);
    }
  }
  __syncthreads();                                         // the shifted waves' last barrier
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The kernel of one output type and direction, for the call's activation.
template <int F32, int MODE>
hipError_t launch_tiles(const FusedArgs &g, dim3 grid, hipStream_t stream) {
  hipError_t e = hipErrorInvalidValue;
  with_act(g.e.act, [&](auto act) {
    e = launch(fused_tile_kernel<F32, MODE, act()>, grid, dim3(kThreads), 0, stream, g);
  });
  return e;
}

}  // namespace tile

// (each in a source file of its own, so that they compile side by side)
hipError_t launch_tiles_bf16(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_bf16_both(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_f32_both(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_f32(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_bf16_grad(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_f32_grad(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_bf16_grad_mul(const FusedArgs &g, dim3 grid, hipStream_t stream);
hipError_t launch_tiles_f32_grad_mul(const FusedArgs &g, dim3 grid, hipStream_t stream);

}  // namespace mx
