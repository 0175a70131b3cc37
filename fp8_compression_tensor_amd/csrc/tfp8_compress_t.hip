// tfp8_compress_t.hip - gfx950 compress of a transpose: codes of x^T with blocks along the rows of
// x, for products whose contraction runs over those rows (the two of a linear layer's backward
// pass), ragged by group where the rows are sorted by expert.
//
// Mathematics: that of k_compress (tfp8_kernels.hip) on every column.  With w = H v over a block
// v of B rows of one column, M = max |w| and E = sum v^2,
//   alpha = clamp(sqrt(T B / E), 2^-126, 2^126), s = alpha M / (448 sqrt(B)), codes E4M3(448 w / M)
// (without the rotation w = v and s = alpha M / 448).  The rotation, the maximum and the energy all
// run down a column, so the transpose is only a matter of which lane holds what.
//
// Layout.  A wavefront takes a block of B rows and 8 C columns.  Lane j + 8 c holds rows
// [R j, R j + R), R = B / 8, of columns [C c, C c + C), read with one load a row: the eight lanes of a
// c read eight rows, the eight c of a row read 8 C consecutive columns (a 128-byte line).  The
// transform is k_compress's: register stages over the R rows, then the butterfly over the lanes j.
// It leaves lane j with R consecutive codes of each column, and the eight lanes of a column store its
// whole block, so no element passes through LDS.  The scales do: a workgroup takes four blocks that
// follow one another in an output row, and stores a column's four alphas and four scales as 16 bytes
// each, where single floats would each cost a write of a line.
//
// Bound by HBM.  [16384, 5120] bfloat16, B = 128 (257 MB with the scales): 53 us, 4.8 TB/s, where a
// large copy reaches 5.0 and k_compress, which reads whole rows, 42 us on the same bytes; before the
// scales went out together and whole blocks lost their per-row conditions, 67 us.  [16384, 5120]
// float32: 92 us, 4.6 TB/s (k_compress 66).  Odd rows and columns: 61 us.  Longer blocks take
// more registers a lane (182 at B = 256, 227 at 512: two wavefronts a SIMD), and at 512 a load of bfloat16
// reads half a line: 60 us at 256 and 78 at 512, float32 91 and 116.  Half as many columns a lane at
// B = 128 (six wavefronts a SIMD instead of four) took 60 us; non-temporal loads and stores were 1-2%
// faster here and 13-17% slower on data that is still in the caches.
#include <math.h>
#include <stdint.h>

#include "../../include/tfp8.h"
#include "tfp8_device.hpp"
#include "tfp8_groups.hpp"
#include "tfp8_host.hpp"

namespace tfp8 {

// Columns a lane holds: 16 bytes of a row, or as many as 512 bytes of a column leave room for.
constexpr int transposed_columns(int B, int es) {
  const int most = 512 / (B / 8 * es);
  return 16 / es < most ? 16 / es : most;
}
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

struct TransposeArgs {
  const void *x;
  int64_t rows, cols, ldx;
  const int64_t *offsets;  // NULL: one group
  int groups;
  int64_t blocks;  // blocks of an output row
  uint32_t tiles;  // column tiles
  float sqrtTB, sqrtTBB, invC;
  uint8_t *codes;
  float *alpha, *scale;
};

// Scales and code multiplier of a block whose 8 lanes hold w in v, with M = max |w| and SS = sum of
// its squares before the rotation (both over the block).  As in k_compress.
template <int R>
__device__ __forceinline__ void column_scales(float (&v)[R], float M, float SS,
                                              const TransposeArgs &p, float &cm, float &alpha,
                                              float &s) {
  if (M >= 0x1p-40f && M <= 0x1p60f) {
    alpha = fminf(fmaxf(p.sqrtTB * __builtin_amdgcn_rsqf(SS), 0x1p-126f), 0x1p126f);
    s = alpha * M * p.invC;
    cm = __fdiv_rn(448.0f, M);
  } else if (M == 0.0f) {
    cm = 0.0f;
    alpha = 1.0f;
    s = 0.0f;
  } else {
    // sum(x^2) leaves float32's range: the same on the block times the power of two that brings
    // M into [1, 2), with the energy of the scaled w (the rotation preserves it)
    const int k = 1 - exponent_of(M);
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = scale2(v[r], k);
    const float Mk = scale2(M, k);
    const float SW = group_sum<8>(sum_squares<R>(v));
    alpha = fminf(fmaxf(scale2(p.sqrtTBB * __builtin_amdgcn_rsqf(SW), k), 0x1p-126f), 0x1p126f);
    s = scale2(alpha * Mk, -k) * p.invC;
    cm = __fdiv_rn(448.0f, Mk);
  }
}

template <int B, bool F32IN, bool ROT>
__global__ __launch_bounds__(256) void k_compress_t(TransposeArgs p) {
  constexpr int ES = F32IN ? 4 : 2;
  constexpr int R = B / 8;
  constexpr int C = transposed_columns(B, ES);
  constexpr int DW = C * ES / 4;  // dwords a lane holds of a row
  const int lane = threadIdx.x & 63;
  const int j = lane & 7, c = lane >> 3;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ float scales[2][8 * C][4];
  // the launch's tiles in eight contiguous parts, one for each XCD, columns first
  const uint32_t per = gridDim.x >> 3, over = gridDim.x & 7, x8 = blockIdx.x & 7;
  const uint32_t bid = x8 * per + (x8 < over ? x8 : over) + (blockIdx.x >> 3);
  const int64_t kb0 = (int64_t)(bid / p.tiles) * 4, kb = kb0 + w;
  const int64_t ct = bid % p.tiles;

  int64_t row0 = 0;
  int rows = 0;
  if (kb < p.blocks) {
    if (p.offsets) {
      const GroupTile g = tile_of_groups(p.offsets, p.groups, p.rows, B, false,
                                         [&](int64_t) { return kb; });
      row0 = g.row0;
      rows = g.rows;
    } else {
      row0 = kb * B;
      rows = (int)(p.rows - row0 < B ? p.rows - row0 : B);
    }
  }
  const int64_t col0 = (ct * 8 + c) * C;
  const int cols = (int)(p.cols - col0 < C ? p.cols - col0 : C);

  // this lane's rows and columns; a whole block of whole chunks takes the loads without conditions
  uint32_t d[R][DW];
  const char *at = (const char *)p.x + ((row0 + R * j) * p.ldx + col0) * ES;
  const int64_t next = p.ldx * ES;
  typedef uint32_t chunk_t __attribute__((ext_vector_type(DW), aligned(ES)));  // at any element
  if (rows == B && __all(cols == C)) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const chunk_t t = *(const chunk_t *)(at + i * next);
#pragma unroll
      for (int k = 0; k < DW; ++k) d[i][k] = t[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int k = 0; k < DW; ++k) d[i][k] = 0;
      if (R * j + i < rows && cols == C) {
        const chunk_t t = *(const chunk_t *)(at + i * next);
#pragma unroll
        for (int k = 0; k < DW; ++k) d[i][k] = t[k];
      } else if (R * j + i < rows) {
#pragma unroll
        for (int k = 0; k < C - 1; ++k)
          if (k < cols) {
            if constexpr (F32IN)
              d[i][k] = ((const uint32_t *)(at + i * next))[k];
            else
              d[i][k / 2] |= (uint32_t)((const uint16_t *)(at + i * next))[k] << (16 * (k & 1));
          }
      }
    }
  }

  const int pj = ROT ? lane_perm<8>(j) : j;
  const float sj = ROT ? lane_sign<8>(j) : 1.0f;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    float v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if constexpr (F32IN)
        v[i] = __uint_as_float(d[i][k]);
      else
        v[i] = __uint_as_float((k & 1) ? d[i][k / 2] & 0xFFFF0000u : d[i][k / 2] << 16);
    }
    const float SS = group_sum<8>(sum_squares<R>(v));
    if constexpr (ROT) {
      fwht_registers<R>(v);
      fwht_lanes<8, R>(v, j);
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) m = fmaxf(m, fabsf(v[i]));
    const float M = group_max<8>(m);
    float cm, alpha, s;
    column_scales<R>(v, M, SS, p, cm, alpha, s);
    cm *= sj;
    if (k < cols && kb < p.blocks) {
      const int64_t o = (col0 + k) * p.blocks + kb;
      uint8_t *to = p.codes + o * B + R * pj;
#pragma unroll
      for (int i = 0; i < R; i += 16) {
        u32x4 q;
#pragma unroll
        for (int t = 0; t < 4; ++t)  // + 0 turns a -0 product into +0
          q[t] = pack_fp8x4(fmaf(v[i + 4 * t], cm, 0.0f), fmaf(v[i + 4 * t + 1], cm, 0.0f),
                            fmaf(v[i + 4 * t + 2], cm, 0.0f), fmaf(v[i + 4 * t + 3], cm, 0.0f));
        *(u32x4 *)(to + i) = q;
      }
    }
    if (j == 0) {
      scales[0][c * C + k][w] = alpha;
      scales[1][c * C + k][w] = s;
    }
  }
  // the scales of a column's four blocks together
  __syncthreads();
  for (int t = threadIdx.x; t < 16 * C; t += 256) {
    const int which = t / (8 * C), i = t % (8 * C);
    const int64_t col = ct * 8 * C + i;
    if (col < p.cols) {
      float *to = (which ? p.scale : p.alpha) + col * p.blocks + kb0;
      const float *from = scales[which][i];
      if (kb0 + 4 <= p.blocks)
        *(f32x4_any *)to = f32x4_any{from[0], from[1], from[2], from[3]};
      else
        for (int k = 0; kb0 + k < p.blocks; ++k) to[k] = from[k];
    }
  }
}

}  // namespace tfp8

namespace {

using namespace tfp8;

template <int B, bool F32, bool ROT>
tfp8_status launch_compress_t(TransposeArgs p, hipStream_t st) {
  constexpr int ES = F32 ? 4 : 2;
  constexpr int C = transposed_columns(B, ES);
  const int64_t tiles = (p.cols + 8 * C - 1) / (8 * C), grid = tiles * ((p.blocks + 3) / 4);
  p.tiles = (uint32_t)tiles;
  if (grid > ((int64_t)1 << 24) - 1) return TFP8_E_SIZE;
  return launch(k_compress_t<B, F32, ROT>, (unsigned)grid, 256, st, p);
}

}  // namespace

extern "C" {

int64_t tfp8_padded_rows(int64_t rows, int32_t groups, int32_t block) {
  if (rows < 0 || rows > TFP8_MAX_N || groups < 1 || groups > TFP8_MAX_GROUPS || block < 1)
    return 0;
  return (rows + (int64_t)groups * (block - 1)) / block * block;
}

tfp8_status tfp8_compress_t(const void *x, tfp8_dtype x_dtype, int64_t rows, int64_t cols,
                            int64_t ldx, const int64_t *offsets, int32_t groups, int32_t block,
                            float target, uint32_t flags, uint8_t *codes, float *alpha,
                            float *scale, void *stream) {
  if (block != 128 && block != 256 && block != 512) return TFP8_E_BLOCK;
  constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
  if (rows < 0 || rows > kMaxRows || cols < 0 || cols > kMaxRows) return TFP8_E_SIZE;
  if (x_dtype != TFP8_BF16 && x_dtype != TFP8_F32) return TFP8_E_DTYPE;
  if (!target_ok(target) || (flags & ~(uint32_t)TFP8_FLAG_NO_ROTATION)) return TFP8_E_ARG;
  if (groups < 1 || groups > TFP8_MAX_GROUPS || (!offsets && groups != 1)) return TFP8_E_ARG;
  if (ldx < cols) return TFP8_E_ARG;
  const int64_t kp = tfp8_padded_rows(rows, groups, block);
  if (cols == 0 || kp == 0) return TFP8_OK;
  if (kp > TFP8_MAX_N / cols || (rows > 0 && ldx > TFP8_MAX_N / rows)) return TFP8_E_SIZE;
  if ((rows > 0 && !x) || !codes || !alpha || !scale) return TFP8_E_NULL;
  const bool f32 = x_dtype == TFP8_F32;
  if (!aligned(x, f32 ? 4 : 2) || !aligned(codes, 16) || !aligned(alpha, 4) ||
      !aligned(scale, 4) || !aligned(offsets, 8))
    return TFP8_E_ALIGN;
  const int64_t nb = cols * (kp / block);
  const Range ins[2] = {range_of(x, rows > 0 ? ((rows - 1) * ldx + cols) * (f32 ? 4 : 2) : 0),
                        range_of(offsets, offsets ? ((int64_t)groups + 1) * 8 : 0)};
  const Range outs[3] = {range_of(codes, cols * kp), range_of(alpha, nb * 4),
                         range_of(scale, nb * 4)};
  for (int i = 0; i < 3; ++i) {
    for (int k = 0; k < 2; ++k)
      if (overlap(outs[i], ins[k])) return TFP8_E_ARG;
    for (int k = i + 1; k < 3; ++k)
      if (overlap(outs[i], outs[k])) return TFP8_E_ARG;
  }
  const bool rot = !(flags & TFP8_FLAG_NO_ROTATION);
  TransposeArgs p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.offsets = offsets;
  p.groups = groups;
  p.blocks = kp / block;
  const double tbb = (double)target * block * (rot ? block : 1);
  p.sqrtTBB = (float)sqrt(tbb);
  p.sqrtTB = (float)sqrt((double)target * block);
  p.invC = (float)(1.0 / (rot ? 448.0 * sqrt((double)block) : 448.0));
  p.codes = codes;
  p.alpha = alpha;
  p.scale = scale;
  hipStream_t st = (hipStream_t)stream;
#define TFP8_CASE(BB)                                                                     \
  case BB:                                                                                \
    return f32 ? (rot ? launch_compress_t<BB, true, true>(p, st)                          \
                      : launch_compress_t<BB, true, false>(p, st))                        \
               : (rot ? launch_compress_t<BB, false, true>(p, st)                         \
                      : launch_compress_t<BB, false, false>(p, st));
  switch (block) {
    TFP8_CASE(128)
    TFP8_CASE(256)
    TFP8_CASE(512)
  }
#undef TFP8_CASE
  return TFP8_E_BLOCK;
}

}  // extern "C"
