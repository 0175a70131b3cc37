// tfp8_groups.hpp - where the rows of a group lie, found on the device from the groups' offsets.
//
// offsets[groups + 1] are device data, so the host launches for the most units the sizes allow and
// each wavefront looks its own up: 64 groups at a time, one per lane, an inclusive scan of their
// unit counts and a ballot.  All 64 lanes must be active.  Whatever the offsets hold, a group's
// rows are clamped to [0, rows) and to a length >= 0, so no row outside the tensor is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tfp8 {

// Rows [lo, hi) of group e; e = groups stands for the rows past the last group.
__device__ __forceinline__ void group_rows(const int64_t *offsets, int groups, int64_t rows, int e,
                                           int &lo, int &hi) {
  int64_t l = offsets[e];
  int64_t h = e < groups ? offsets[e + 1] : rows;
  l = l < 0 ? 0 : (l > rows ? rows : l);
  h = h < l ? l : (h > rows ? rows : h);
  lo = (int)l;
  hi = (int)h;
}

__device__ __forceinline__ int wave_inclusive_sum(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct GroupTile {
  int row0, rows;  // first row and number of rows of the tile; rows = 0: there is no such tile
  int group;
};

// 64 groups, one a lane: their rows, their tiles of at most `size` rows, and the sum of these up to
// the lane's own (of groups that do not overlap; the sum of others may wrap).
struct GroupScan {
  int lo, hi, tiles, incl;
};
__device__ __forceinline__ GroupScan scan_groups(const int64_t *offsets, int groups, int64_t rows,
                                                 int size, int g0, int last) {
  const int lane = threadIdx.x & 63, e = g0 + lane;
  GroupScan s{0, 0, 0, 0};
  if (e <= last) group_rows(offsets, groups, rows, e, s.lo, s.hi);
  s.tiles = (int)(((int64_t)(s.hi - s.lo) + size - 1) / size);
  s.incl = wave_inclusive_sum(s.tiles, lane);
  return s;
}

// A tile of at most `size` rows, counting the tiles of group 0, 1, ... up to group `last` (last =
// groups counts the rows past the last group as one more group): the one that pick(how many there
// are) names.
template <class PICK>
__device__ __forceinline__ GroupTile tile_of_groups(const int64_t *offsets, int groups,
                                                    int64_t rows, int size, int last, PICK pick) {
  GroupScan s = scan_groups(offsets, groups, rows, size, 0, last);
  int64_t all = __builtin_amdgcn_readfirstlane(__shfl(s.incl, 63));
  for (int g0 = 64; g0 <= last; g0 += 64)
    all += __builtin_amdgcn_readfirstlane(
        __shfl(scan_groups(offsets, groups, rows, size, g0, last).incl, 63));
  const int64_t idx = pick(all);
  int64_t before = 0;
  for (int g0 = 0;;) {
    const uint64_t past = __ballot(before + s.incl > idx);
    if (past) {
      const int f = __builtin_ctzll(past);
      const int tiles = __builtin_amdgcn_readfirstlane(__shfl(s.tiles, f));
      const int t =
          __builtin_amdgcn_readfirstlane((int)(idx - before) - (__shfl(s.incl, f) - tiles));
      const int l = __shfl(s.lo, f), h = __shfl(s.hi, f);
      if ((uint32_t)t >= (uint32_t)tiles) break;  // wrapped sums
      GroupTile r;
      r.row0 = __builtin_amdgcn_readfirstlane(l + t * size);
      r.rows = __builtin_amdgcn_readfirstlane(h - r.row0 < size ? h - r.row0 : size);
      r.group = __builtin_amdgcn_readfirstlane(g0 + f);
      return r;
    }
    before += __builtin_amdgcn_readfirstlane(__shfl(s.incl, 63));
    g0 += 64;
    if (g0 > last) break;
    s = scan_groups(offsets, groups, rows, size, g0, last);
  }
  return GroupTile{0, 0, 0};
}

struct GroupSpan {
  int64_t unit0, units;
};

// Where group e lies in a padded row: its first unit of `size` rows and how many it has.
__device__ __forceinline__ GroupSpan span_of_group(const int64_t *offsets, int groups,
                                                   int64_t rows, int size, int e) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 <= e; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < groups) group_rows(offsets, groups, rows, g, lo, hi);
    const int units = (int)(((int64_t)(hi - lo) + size - 1) / size);
    const int incl = wave_inclusive_sum(units, lane);
    if (e < g0 + 64) {
      const int mine = __shfl(units, e - g0);
      GroupSpan s;
      s.units = __builtin_amdgcn_readfirstlane(mine);
      s.unit0 = before + __builtin_amdgcn_readfirstlane(__shfl(incl, e - g0) - mine);
      return s;
    }
    before += __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
  }
  return GroupSpan{0, 0};
}

}  // namespace tfp8
