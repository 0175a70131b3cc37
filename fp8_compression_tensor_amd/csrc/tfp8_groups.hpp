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

// The idx-th tile of at most `size` rows, counting the tiles of group 0, 1, ... up to group
// `last` (last = groups counts the rows past the last group as one more group).
__device__ __forceinline__ GroupTile tile_of_groups(const int64_t *offsets, int groups,
                                                    int64_t rows, int size, int64_t idx,
                                                    int last) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 <= last; g0 += 64) {
    const int e = g0 + lane;
    int lo = 0, hi = 0;
    if (e <= last) group_rows(offsets, groups, rows, e, lo, hi);
    const int tiles = (int)(((int64_t)(hi - lo) + size - 1) / size);
    const int incl = wave_inclusive_sum(tiles, lane);  // <= 64 * 2^31 / size
    const uint64_t past = __ballot(before + incl > idx);
    if (past) {
      const int f = __builtin_ctzll(past);
      const int t = (int)(idx - before) - (__shfl(incl, f) - __shfl(tiles, f));
      const int l = __shfl(lo, f), h = __shfl(hi, f);
      GroupTile r;
      r.row0 = __builtin_amdgcn_readfirstlane(l + t * size);
      r.rows = __builtin_amdgcn_readfirstlane(h - r.row0 < size ? h - r.row0 : size);
      r.group = __builtin_amdgcn_readfirstlane(g0 + f);
      return r;
    }
    before += __shfl(incl, 63);
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
