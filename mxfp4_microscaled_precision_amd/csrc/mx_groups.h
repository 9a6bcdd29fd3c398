// Groups of rows (the rows of one expert after another) on the device: where a
// group begins, and which group a tile, a block or a slice of a launch is in.
//
// The groups are given by their ends, ends[e] = the row behind group e's last,
// which only the device knows. An end below an earlier one counts as that one
// and an end past the last row as the last row, so whatever the array holds,
// groups are ranges of rows that follow one another, [0, rows) at most. Equal
// groups (ends == nullptr) are `each` rows long.
//
// A wave looks 64 ends up at once: a maximum scan makes ranges of them, a sum
// scan counts tiles or slices, and a ballot finds the group. For up to 64
// groups that is one load and some twenty VALU instructions a tile, so no launch of
// its own prepares a table and nothing has to be stored between launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Inclusive scans over the 64 lanes in six DPP steps (within rows of 16 by 1,
// 2, 4, 8, then across them); lanes without a partner keep what they hold
// (values are >= 0, so a partner of 0 changes nothing).
__device__ __forceinline__ int scan_add(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row 15's last lane to the next row
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to the upper half
  return v;
}

__device__ __forceinline__ int scan_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}

// Group g: rows [first, last), and how many units (tiles, slices) the groups
// before it have. g == groups: behind the last group (first == last).
struct Group {
  int g, first, last, before;
};

// What a group's rows [first, last) count as: 128-row slices, or tiles of
// TILE rows from the multiple of ALIGN at or below its first row.
struct CountSlices {
  __device__ __forceinline__ int operator()(int first, int last) const {
    return (last - first + 127) >> 7;
  }
};
template <int TILE, int ALIGN>
struct CountTiles {
  __device__ __forceinline__ int operator()(int first, int last) const {
    return last > first ? (last - (first & ~(ALIGN - 1)) + TILE - 1) / TILE : 0;
  }
};

// The group that holds unit `unit` (BY_UNIT), or group number `unit` (else).
// Every lane of the wave must be active; the result is wave-uniform.
template <bool BY_UNIT, typename Count>
__device__ __forceinline__ Group find_group(const int32_t *ends, int groups, int rows, int each,
                                            int unit, Count count) {
  const int lane = (int)__lane_id();
  int row = 0, before = 0;                           // where the groups seen so far end
  for (int base = 0; base < groups; base += 64) {
    const int e = base + lane;
    int last = 0;
    if (e < groups) last = ends ? min(max(ends[e], 0), rows) : (int)min((int64_t)(e + 1) * each, (int64_t)rows);
    last = max(scan_max(last), row);
    int first = __builtin_amdgcn_update_dpp(row, last, 0x138, 0xF, 0xF, false);   // the lane before
    const int units = scan_add(e < groups ? count(first, last) : 0) + before;
    const uint64_t past = __ballot(BY_UNIT ? units > unit : e >= unit);
    if (past) {
      const int l = __builtin_ctzll(past);
      if (base + l < groups) {
        const int prev = l ? __builtin_amdgcn_readlane(units, l ? l - 1 : 0) : before;
        return Group{base + l, __builtin_amdgcn_readlane(first, l),
                     __builtin_amdgcn_readlane(last, l), prev};
      }
    }
    row = __builtin_amdgcn_readlane(last, 63);
    before = __builtin_amdgcn_readlane(units, 63);
  }
  return Group{groups, row, row, before};
}

}  // namespace mx
