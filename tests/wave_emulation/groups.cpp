// csrc/tfp8_groups.hpp on the host: C entry points for tests/test_groups.py.
#include "hip/hip_runtime.h"

#include "../../fp8_compression_tensor_amd/csrc/tfp8_groups.hpp"

namespace {

const int64_t *g_offsets;
int64_t g_rows, g_idx;
int g_groups, g_size;
bool g_all_rows;
int64_t out[64][4];

void one_tile() {
  int64_t there = -1;
  const tfp8::GroupTile t =
      tfp8::tile_of_groups(g_offsets, g_groups, g_rows, g_size, g_all_rows, [&](int64_t n) {
        there = n;
        return g_idx;
      });
  int64_t *o = out[threadIdx.x];
  o[0] = t.row0, o[1] = t.rows, o[2] = t.group, o[3] = there;
}

void one_span() {
  const tfp8::GroupSpan s =
      tfp8::span_of_group(g_offsets, g_groups, g_rows, g_size, (int)g_idx);
  int64_t *o = out[threadIdx.x];
  o[0] = s.unit0, o[1] = s.units, o[2] = o[3] = 0;
}

// 0, and what all lanes agree on; -1 where they do not
int result(bool met, int64_t *to) {
  for (int i = 1; i < 64; ++i)
    for (int k = 0; k < 4; ++k) met &= out[i][k] == out[0][k];
  for (int k = 0; k < 4; ++k) to[k] = out[0][k];
  return met ? 0 : -1;
}

void set(const int64_t *offsets, int groups, int64_t rows, int size, int64_t idx) {
  g_offsets = offsets, g_groups = groups, g_rows = rows, g_size = size, g_idx = idx;
}

}  // namespace

extern "C" int tile(const int64_t *offsets, int groups, int64_t rows, int size, int all_rows,
                    int64_t idx, int64_t *to) {
  set(offsets, groups, rows, size, idx);
  g_all_rows = all_rows;
  return result(wave::run(one_tile), to);
}

extern "C" int span(const int64_t *offsets, int groups, int64_t rows, int size, int e,
                    int64_t *to) {
  set(offsets, groups, rows, size, e);
  return result(wave::run(one_span), to);
}
