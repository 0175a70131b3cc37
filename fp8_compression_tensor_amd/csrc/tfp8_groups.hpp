// tfp8_groups.hpp - where the rows of a group lie, found on the device from the groups' offsets.
//
// offsets[groups + 1] are device data, so the host launches for the most units the sizes allow and
// each wavefront looks its own up: 64 groups at a time, one per lane, an inclusive scan of their
// unit counts and a ballot.  All 64 lanes must be active.  Whatever the offsets hold, they are taken
// as clamped to [0, rows] and to the largest before them, so that groups never overlap, every
// row is in one group at most, and no row outside the tensor is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tfp8 {

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
  int group;       // -1: the rows are of no group
};

// 64 groups from g0 on, one a lane: their rows [lo, hi), their tiles of at most `size` rows, and the
// sum of these up to the lane's own.  Group -1 stands for the rows before the first group, and
// group `groups` for those past the last.  `reach` is where the groups before g0 end.
struct GroupScan {
  int lo, hi, tiles, incl;
};
__device__ __forceinline__ GroupScan scan_groups(const int64_t *offsets, int groups, int64_t rows,
                                                 int size, int g0, int last, int reach) {
  const int lane = threadIdx.x & 63, e = g0 + lane;
  GroupScan s{0, 0, 0, 0};
  if (e <= last) {
    const int64_t l = e < 0 ? 0 : offsets[e], h = e < groups ? offsets[e + 1] : rows;
    s.lo = (int)(l < 0 ? 0 : (l > rows ? rows : l));
    s.hi = (int)(h < 0 ? 0 : (h > rows ? rows : h));
  }
  if (__ballot(e <= last && (s.hi < s.lo || s.lo < reach))) {  // descending: the largest so far
    int most = s.lo > s.hi ? s.lo : s.hi;
    most = most > reach ? most : reach;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(most, d);
      if (lane >= d && o > most) most = o;
    }
    const int before = __shfl_up(most, 1);
    s.lo = s.lo > reach ? s.lo : reach;
    if (lane > 0 && before > s.lo) s.lo = before;
    s.hi = most;
  }
  if (e <= last) s.tiles = (int)(((int64_t)(s.hi - s.lo) + size - 1) / size);
  s.incl = wave_inclusive_sum(s.tiles, lane);
  return s;
}

// A tile of at most `size` rows, counting the tiles of group 0, 1, ... up to the last (all_rows: of
// group -1 to group `groups`, so that every row is in a tile): the one that pick(how many there are)
// names.
template <class PICK>
__device__ __forceinline__ GroupTile tile_of_groups(const int64_t *offsets, int groups,
                                                    int64_t rows, int size, bool all_rows,
                                                    PICK pick) {
  const int first = all_rows ? -1 : 0, last = all_rows ? groups : groups - 1;
  GroupScan s = scan_groups(offsets, groups, rows, size, first, last, 0);
  const auto total = [](const GroupScan &x) {
    return __builtin_amdgcn_readfirstlane(__shfl(x.incl, 63));
  };
  const auto reach = [](const GroupScan &x) {
    return __builtin_amdgcn_readfirstlane(__shfl(x.hi, 63));
  };
  int64_t all = total(s);
  GroupScan t = s;
  for (int g0 = first + 64; g0 <= last; g0 += 64) {
    t = scan_groups(offsets, groups, rows, size, g0, last, reach(t));
    all += total(t);
  }
  const int64_t idx = pick(all);
  int64_t before = 0;
  for (int g0 = first; idx < all;) {
    const uint64_t past = __ballot(before + s.incl > idx);
    if (past) {
      const int f = __builtin_ctzll(past);
      const int at =
          __builtin_amdgcn_readfirstlane((int)(idx - before) - (__shfl(s.incl, f) - __shfl(s.tiles, f)));
      const int l = __shfl(s.lo, f), h = __shfl(s.hi, f);
      GroupTile r;
      r.row0 = __builtin_amdgcn_readfirstlane(l + at * size);
      r.rows = __builtin_amdgcn_readfirstlane(h - r.row0 < size ? h - r.row0 : size);
      r.group = g0 + f < groups ? g0 + f : -1;
      return r;
    }
    before += total(s);
    g0 += 64;
    if (g0 > last) break;
    s = scan_groups(offsets, groups, rows, size, g0, last, reach(s));
  }
  return GroupTile{0, 0, -1};
}

struct GroupSpan {
  int64_t unit0, units;
};

// Where group e lies in a padded row: its first unit of `size` rows and how many it has.
__device__ __forceinline__ GroupSpan span_of_group(const int64_t *offsets, int groups,
                                                   int64_t rows, int size, int e) {
  int64_t before = 0;
  int reach = 0;
  for (int g0 = 0; g0 <= e; g0 += 64) {
    const GroupScan s = scan_groups(offsets, groups, rows, size, g0, groups - 1, reach);
    if (e < g0 + 64) {
      const int mine = __shfl(s.tiles, e - g0);
      GroupSpan r;
      r.units = __builtin_amdgcn_readfirstlane(mine);
      r.unit0 = before + __builtin_amdgcn_readfirstlane(__shfl(s.incl, e - g0) - mine);
      return r;
    }
    before += __builtin_amdgcn_readfirstlane(__shfl(s.incl, 63));
    reach = __builtin_amdgcn_readfirstlane(__shfl(s.hi, 63));
  }
  return GroupSpan{0, 0};
}

}  // namespace tfp8
