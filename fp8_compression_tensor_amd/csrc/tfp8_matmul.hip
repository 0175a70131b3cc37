// tfp8_matmul.hip - gfx950 products of compressed operands: C = A^ B^T where A^ and B^ are what
// the codes of A[M, K] and B[N, K] stand for, dense, grouped by rows, and grouped along the
// contraction.
//
// Mathematics.  Both operands are compressed in blocks along K with the same rotation, so a
// block of a row is a^ = H u_a / sqrt(B), u_a = r_a dec(q_a), r_a = s_a / alpha_a (without the
// rotation a^ = u_a).  H / sqrt(B) is orthogonal: a^ . b^ = u_a . u_b, and
//   C[m][n] = sum over blocks of r_a[m] r_b[n] sum_k dec(qa[m][k]) dec(qb[n][k]).
// The inner sum is what the matrix cores compute on the codes as they are; no Hadamard, no
// decompressed copy.  Each 128-deep partial tile is scaled by r_a r_b and added in float32.
#include <math.h>
#include <stdint.h>

#include "../../include/tfp8.h"
#include "tfp8_device.hpp"
#include "tfp8_groups.hpp"
#include "tfp8_host.hpp"

namespace tfp8 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kStep = 128;  // contraction depth of one matrix instruction

// A compressed operand: rows of codes `ld` bytes apart, rows of scales `lds` floats apart, and for
// a stack of them (experts) the distance from one to the next.
struct Operand {
  const uint8_t *codes;
  const float *alpha, *scale;
  int64_t ld, lds;
  int64_t next, next_s;
};

enum : int { kDense = 0, kGroupedRows = 1, kGroupedDepth = 2 };

struct ProductArgs {
  Operand a, b;
  int64_t m, n;          // rows of A (all groups together, kGroupedRows) and of B
  int64_t steps;         // kStep-deep steps along a row
  int shift;             // log2(block / kStep): steps 2^shift s .. share a scale
  const int64_t *offsets;
  int groups;
  int64_t rows;          // kGroupedDepth: rows of the uncompressed operands
  void *out;
  int64_t ldc, next_c;
  int mtiles, ntiles;
};

// 16 x 16 partial tile over 128 codes: D[4 q + i][l & 15], q = l >> 4, of rows of x by rows of y.
// Lane l gives 32 codes of row l & 15 of each; both take the same codes of the row for the same
// lane group, so which of the 128 they are does not matter.
//
// The 8-bit matrix instructions add eight products at a time as fixed point numbers, with 14 bits
// from the largest one's down (measured: beside a product of 2^16, one of 2^3 counts and one of
// 2^2 does not, whatever the instruction's shape), and the eights in float32.  That is 1.4e-5 of
// the result for codes as compress makes them, a hundredth of a bfloat16 output's rounding, so
// bfloat16 outputs use them.  float32 outputs widen the codes to bfloat16, which is exact, and use
// the bfloat16 instructions, whose sums are float32 throughout (1e-8 on the same codes), at half
// the rate.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool WIDE>
struct Fragment;
template <>
struct Fragment<false> {
  i32x8 v;
};
template <>
struct Fragment<true> {
  bf16x8 v[4];  // 8 codes each
};

template <bool WIDE>
__device__ __forceinline__ Fragment<WIDE> make_fragment(u32x4 lo, u32x4 hi) {
  Fragment<WIDE> f;
  if constexpr (WIDE) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t d0 = t < 2 ? lo[2 * t] : hi[2 * t - 4];
      const uint32_t d1 = t < 2 ? lo[2 * t + 1] : hi[2 * t - 3];
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, false);
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, true);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, false);
      const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, true);
      f.v[t] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
  } else {
    f.v = i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
  return f;
}

__device__ __forceinline__ f32x4 mfma_codes(const Fragment<false> &x, const Fragment<false> &y) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_codes(const Fragment<true> &x, const Fragment<true> &y) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < 4; ++t)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v[t], y.v[t], d, 0, 0, 0);
  return d;
}

template <bool F32OUT>
__device__ __forceinline__ void store_values(void *out, int64_t at, const f32x4 v, int valid,
                                             bool wide) {
  if constexpr (F32OUT) {
    float *o = (float *)out + at;
    if (wide && valid >= 4) {
      *(f32x4 *)o = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < valid) o[i] = v[i];
    }
  } else {
    __bf16 *o = (__bf16 *)out + at;
    __bf16 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = (__bf16)v[i];
    if (wide && valid >= 4) {
      u32x2 w;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, h[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, h[2 * i + 1]) << 16);
      *(u32x2 *)o = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < valid) o[i] = h[i];
    }
  }
}

template <int BM, int BN, int WM, int WN, int MODE, bool F32OUT>
__device__ __forceinline__ void matmul_tile(const ProductArgs &p) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;
  constexpr int ROWS = BM + BN;
  constexpr int NT = 64 * NW;
  constexpr int LOADS = ROWS / 8 / NW;  // 1 KB loads of a wavefront a step (8 rows each)
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole loads of one operand");
  constexpr int SC = (ROWS + NT - 1) / NT;  // rows whose scales a thread prepares
  __shared__ alignas(1024) uint8_t tile[2][ROWS * kStep];
  __shared__ float rsc[2][ROWS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, l16 = lane & 15;
  const int wm = w / WN, wn = w % WN;

  // the tile of this workgroup
  int64_t bid = blockIdx.x;
  int64_t m0, m1, n0, s0 = 0, s1 = p.steps;
  Operand a = p.a, b = p.b;
  char *out = (char *)p.out;
  constexpr int ES = F32OUT ? 4 : 2;
  if constexpr (MODE == kGroupedDepth) {
    const int per = p.mtiles * p.ntiles;
    const int e = (int)(bid / per);
    bid -= (int64_t)e * per;
    const GroupSpan g = span_of_group(p.offsets, p.groups, p.rows, kStep << p.shift, e);
    s0 = g.unit0 << p.shift;
    s1 = (g.unit0 + g.units) << p.shift;
    s1 = s1 < p.steps ? s1 : p.steps;
    s0 = s0 < s1 ? s0 : s1;
    out += (int64_t)e * p.next_c * ES;
  }
  const int mt = (int)(bid / p.ntiles), nt = (int)(bid % p.ntiles);
  n0 = (int64_t)nt * BN;
  if constexpr (MODE == kGroupedRows) {
    const GroupTile g = tile_of_groups(p.offsets, p.groups, p.m, BM, mt, p.groups);
    if (g.rows <= 0) return;
    m0 = g.row0;
    m1 = g.row0 + g.rows;
    if (g.group == p.groups) {  // rows past the last group: zeros
      s1 = 0;
    } else {
      b.codes += (int64_t)g.group * b.next;
      b.alpha += (int64_t)g.group * b.next_s;
      b.scale += (int64_t)g.group * b.next_s;
    }
  } else {
    m0 = (int64_t)mt * BM;
    m1 = m0 + BM < p.m ? m0 + BM : p.m;
  }
  const int mv = (int)(m1 - m0);
  const int nv = (int)(n0 + BN < p.n ? BN : p.n - n0);

  // Loads.  A wavefront's load instruction fills 8 rows of 128 bytes of LDS, lane i the i-th 16
  // bytes; it takes them from chunk (i & 7) ^ (row & 7) of its row, so that the lanes that read
  // a column of fragments touch all banks.  Rows past the operand's end read as zeros (the
  // descriptor's bound).
  const auto ra = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.codes + m0 * a.ld), 0, (int)((mv - 1) * a.ld + p.steps * kStep), 0x00020000);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(b.codes + n0 * b.ld), 0, (int)((nv - 1) * b.ld + p.steps * kStep), 0x00020000);
  int voff[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int row = (i * NW + w) * 8 + (lane >> 3);
    const int chunk = (lane & 7) ^ (row & 7);
    voff[i] = row < BM ? row * (int)a.ld + chunk * 16 : (row - BM) * (int)b.ld + chunk * 16;
  }
  auto load_step = [&](int64_t s, int stage) {
    const int k0 = (int)(s * kStep);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      lds_void *to = (lds_void *)&tile[stage][(i * NW + w) * 1024];
      if (i < BM / 8 / NW)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to, 16, voff[i], k0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to, 16, voff[i], k0, 0, 0);
    }
  };
  // scales: thread t prepares r = scale / alpha of row t (A's rows, then B's)
  const float *sp[SC], *ap[SC];
#pragma unroll
  for (int i = 0; i < SC; ++i) {
    int row = tid + i * NT;
    row = row < ROWS ? row : ROWS - 1;
    const bool isa = row < BM;
    int64_t rr = isa ? row : row - BM;
    const int64_t last = (isa ? mv : nv) - 1;
    rr = rr < last ? rr : last;
    const int64_t at = isa ? (m0 + rr) * a.lds : (n0 + rr) * b.lds;
    sp[i] = (isa ? a.scale : b.scale) + at;
    ap[i] = (isa ? a.alpha : b.alpha) + at;
  }
  float sv[SC], av[SC];
  auto load_scales = [&](int64_t s) {
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      sv[i] = sp[i][s >> p.shift];
      av[i] = ap[i][s >> p.shift];
    }
  };
  auto put_scales = [&](int stage) {
#pragma unroll
    for (int i = 0; i < SC; ++i)
      if (tid + i * NT < ROWS) rsc[stage][tid + i * NT] = __fdiv_rn(sv[i], av[i]);
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (s0 < s1) {
    load_step(s0, 0);
    load_scales(s0);
  }
  for (int64_t s = s0; s < s1; ++s) {
    const int stage = (int)(s - s0) & 1;
    put_scales(stage);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < s1) {
      load_step(s + 1, stage ^ 1);
      load_scales(s + 1);
    }
    const uint8_t *tl = tile[stage];
    auto fragment = [&](int row) {
      const int at = row * kStep + (((2 * q) ^ (row & 7)) << 4);
      return make_fragment<F32OUT>(*(const u32x4 *)(tl + at), *(const u32x4 *)(tl + (at ^ 16)));
    };
    Fragment<F32OUT> fb[TN];
    f32x4 rbv[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int row = BM + (wn * TN + j) * 16;
      fb[j] = fragment(row + l16);
      rbv[j] = *(const f32x4 *)&rsc[stage][row + 4 * q];
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = (wm * TM + i) * 16 + l16;
      const Fragment<F32OUT> fa = fragment(row);
      const float rav = rsc[stage][row];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const f32x4 part = mfma_codes(fb[j], fa);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(part[k], rav * rbv[j][k], acc[i][j][k]);
      }
    }
  }

  const bool wide = ((uintptr_t)out % (4 * ES) == 0) && (p.ldc % 4 == 0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = (wm * TM + i) * 16 + l16;
    if (row < mv) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int col = (wn * TN + j) * 16 + 4 * q;
        store_values<F32OUT>(out, (m0 + row) * p.ldc + n0 + col, acc[i][j], nv - col, wide);
      }
    }
  }
}

// The kernel only calls the function above: the host's pass over a kernel's own body does not know
// the buffer descriptors' type.
template <int BM, int BN, int WM, int WN, int MODE, bool F32OUT>
__global__ __launch_bounds__(64 * WM * WN) void k_matmul_tile(ProductArgs p) {
  matmul_tile<BM, BN, WM, WN, MODE, F32OUT>(p);
}

}  // namespace tfp8

namespace {

using namespace tfp8;

bool product_block_ok(int32_t block) { return block == 128 || block == 256 || block == 512; }

template <int MODE, bool F32OUT>
tfp8_status launch_product(ProductArgs p, hipStream_t st) {
  constexpr int BM = 128, BN = 128;
  int64_t mt = (p.m + BM - 1) / BM;
  if (MODE == kGroupedRows) mt = (p.m + (int64_t)(p.groups + 1) * (BM - 1)) / BM;
  const int64_t nt = (p.n + BN - 1) / BN;
  int64_t grid = mt * nt;
  if (MODE == kGroupedDepth) grid *= p.groups;
  if (grid > (((int64_t)1 << 32) - 1) / 256) return TFP8_E_SIZE;
  p.mtiles = (int)mt;
  p.ntiles = (int)nt;
  return launch(k_matmul_tile<BM, BN, 2, 2, MODE, F32OUT>, (unsigned)grid, 256, st, p);
}

template <int MODE>
tfp8_status launch_product(const ProductArgs &p, bool f32, hipStream_t st) {
  return f32 ? launch_product<MODE, true>(p, st) : launch_product<MODE, false>(p, st);
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;  // rows and columns of one operand
constexpr int64_t kMaxLd = (int64_t)1 << 22;          // codes of a row: a tile's offsets fit 31 bits

// Checks of one operand [rows, k] (count of them, `next` bytes apart): strides, pointers.
tfp8_status operand_sizes(int64_t rows, int64_t k, int32_t block, int64_t ld, int64_t lds) {
  if (rows < 0 || rows > kMaxRows || k < 0 || k > kMaxLd || k % block != 0) return TFP8_E_SIZE;
  if (ld > kMaxLd || lds > kMaxLd) return TFP8_E_SIZE;
  if (ld < k || lds < k / block) return TFP8_E_ARG;
  return TFP8_OK;
}
bool operand_aligned(const uint8_t *codes, const float *alpha, const float *scale, int64_t ld) {
  return aligned(codes, 16) && aligned(alpha, 4) && aligned(scale, 4) && ld % 16 == 0;
}
struct Spans {
  Range r[6];
  int count = 0;
  void add(const void *p, int64_t bytes) { r[count++] = range_of(p, bytes); }
  void add_operand(const uint8_t *codes, const float *alpha, const float *scale, int64_t rows,
                   int64_t k, int32_t block, int64_t ld, int64_t lds) {
    if (rows == 0 || k == 0) return;
    add(codes, (rows - 1) * ld + k);
    add(alpha, ((rows - 1) * lds + k / block) * 4);
    add(scale, ((rows - 1) * lds + k / block) * 4);
  }
  bool meets(Range o) const {
    for (int i = 0; i < count; ++i)
      if (overlap(o, r[i])) return true;
    return false;
  }
};
int log2_of(int32_t block) { return block == 128 ? 0 : block == 256 ? 1 : 2; }

}  // namespace

extern "C" {

tfp8_status tfp8_matmul(const uint8_t *a_codes, int64_t a_ld, const float *a_alpha,
                        const float *a_scale, int64_t a_lds, const uint8_t *b_codes, int64_t b_ld,
                        const float *b_alpha, const float *b_scale, int64_t b_lds, int64_t m,
                        int64_t n, int64_t k, int32_t block, void *out, tfp8_dtype out_dtype,
                        int64_t ldc, void *stream) {
  if (!product_block_ok(block)) return TFP8_E_BLOCK;
  tfp8_status st = operand_sizes(m, k, block, a_ld, a_lds);
  if (st == TFP8_OK) st = operand_sizes(n, k, block, b_ld, b_lds);
  if (st != TFP8_OK) return st;
  if (out_dtype != TFP8_BF16 && out_dtype != TFP8_F32) return TFP8_E_DTYPE;
  if (ldc < n) return TFP8_E_ARG;
  if (m == 0 || n == 0) return TFP8_OK;
  if (ldc > TFP8_MAX_N / m) return TFP8_E_SIZE;
  const bool f32 = out_dtype == TFP8_F32;
  if (!out || (k > 0 && (!a_codes || !a_alpha || !a_scale || !b_codes || !b_alpha || !b_scale)))
    return TFP8_E_NULL;
  if ((k > 0 && (!operand_aligned(a_codes, a_alpha, a_scale, a_ld) ||
                 !operand_aligned(b_codes, b_alpha, b_scale, b_ld))) ||
      !aligned(out, f32 ? 4 : 2))
    return TFP8_E_ALIGN;
  Spans in;
  in.add_operand(a_codes, a_alpha, a_scale, m, k, block, a_ld, a_lds);
  in.add_operand(b_codes, b_alpha, b_scale, n, k, block, b_ld, b_lds);
  if (in.meets(range_of(out, ((m - 1) * ldc + n) * (f32 ? 4 : 2)))) return TFP8_E_ARG;
  ProductArgs p{};
  p.a = Operand{a_codes, a_alpha, a_scale, a_ld, a_lds, 0, 0};
  p.b = Operand{b_codes, b_alpha, b_scale, b_ld, b_lds, 0, 0};
  p.m = m;
  p.n = n;
  p.steps = k / kStep;
  p.shift = log2_of(block);
  p.out = out;
  p.ldc = ldc;
  return launch_product<kDense>(p, f32, (hipStream_t)stream);
}

tfp8_status tfp8_matmul_grouped(const uint8_t *a_codes, int64_t a_ld, const float *a_alpha,
                                const float *a_scale, int64_t a_lds, const uint8_t *b_codes,
                                int64_t b_ld, const float *b_alpha, const float *b_scale,
                                int64_t b_lds, const int64_t *offsets, int32_t groups, int64_t m,
                                int64_t n, int64_t k, int32_t block, void *out,
                                tfp8_dtype out_dtype, int64_t ldc, void *stream) {
  if (!product_block_ok(block)) return TFP8_E_BLOCK;
  if (groups < 1 || groups > TFP8_MAX_GROUPS) return TFP8_E_ARG;
  tfp8_status st = operand_sizes(m, k, block, a_ld, a_lds);
  if (st == TFP8_OK) st = operand_sizes(n, k, block, b_ld, b_lds);
  if (st != TFP8_OK) return st;
  if (n > kMaxRows / groups) return TFP8_E_SIZE;
  if (out_dtype != TFP8_BF16 && out_dtype != TFP8_F32) return TFP8_E_DTYPE;
  if (ldc < n) return TFP8_E_ARG;
  if (m == 0 || n == 0) return TFP8_OK;
  if (ldc > TFP8_MAX_N / m) return TFP8_E_SIZE;
  const bool f32 = out_dtype == TFP8_F32;
  if (!out || !offsets ||
      (k > 0 && (!a_codes || !a_alpha || !a_scale || !b_codes || !b_alpha || !b_scale)))
    return TFP8_E_NULL;
  if ((k > 0 && (!operand_aligned(a_codes, a_alpha, a_scale, a_ld) ||
                 !operand_aligned(b_codes, b_alpha, b_scale, b_ld))) ||
      !aligned(out, f32 ? 4 : 2) || !aligned(offsets, 8))
    return TFP8_E_ALIGN;
  Spans in;
  in.add_operand(a_codes, a_alpha, a_scale, m, k, block, a_ld, a_lds);
  in.add_operand(b_codes, b_alpha, b_scale, (int64_t)groups * n, k, block, b_ld, b_lds);
  const Range o = range_of(out, ((m - 1) * ldc + n) * (f32 ? 4 : 2));
  if (in.meets(o) || overlap(o, range_of(offsets, ((int64_t)groups + 1) * 8))) return TFP8_E_ARG;
  ProductArgs p{};
  p.a = Operand{a_codes, a_alpha, a_scale, a_ld, a_lds, 0, 0};
  p.b = Operand{b_codes, b_alpha, b_scale, b_ld, b_lds, n * b_ld, n * b_lds};
  p.m = m;
  p.n = n;
  p.steps = k / kStep;
  p.shift = log2_of(block);
  p.offsets = offsets;
  p.groups = groups;
  p.out = out;
  p.ldc = ldc;
  return launch_product<kGroupedRows>(p, f32, (hipStream_t)stream);
}

tfp8_status tfp8_matmul_grouped_t(const uint8_t *a_codes, int64_t a_ld, const float *a_alpha,
                                  const float *a_scale, int64_t a_lds, const uint8_t *b_codes,
                                  int64_t b_ld, const float *b_alpha, const float *b_scale,
                                  int64_t b_lds, const int64_t *offsets, int32_t groups,
                                  int64_t rows, int64_t m, int64_t n, int32_t block, void *out,
                                  tfp8_dtype out_dtype, void *stream) {
  if (!product_block_ok(block)) return TFP8_E_BLOCK;
  if (groups < 1 || groups > TFP8_MAX_GROUPS) return TFP8_E_ARG;
  if (rows < 0 || rows > kMaxRows) return TFP8_E_SIZE;
  const int64_t k = tfp8_padded_rows(rows, groups, block);
  tfp8_status st = operand_sizes(m, k, block, a_ld, a_lds);
  if (st == TFP8_OK) st = operand_sizes(n, k, block, b_ld, b_lds);
  if (st != TFP8_OK) return st;
  if (out_dtype != TFP8_BF16 && out_dtype != TFP8_F32) return TFP8_E_DTYPE;
  if (m == 0 || n == 0) return TFP8_OK;
  if (m * n > TFP8_MAX_N / groups) return TFP8_E_SIZE;
  const bool f32 = out_dtype == TFP8_F32;
  if (!out || !offsets ||
      (k > 0 && (!a_codes || !a_alpha || !a_scale || !b_codes || !b_alpha || !b_scale)))
    return TFP8_E_NULL;
  if ((k > 0 && (!operand_aligned(a_codes, a_alpha, a_scale, a_ld) ||
                 !operand_aligned(b_codes, b_alpha, b_scale, b_ld))) ||
      !aligned(out, f32 ? 4 : 2) || !aligned(offsets, 8))
    return TFP8_E_ALIGN;
  Spans in;
  in.add_operand(a_codes, a_alpha, a_scale, m, k, block, a_ld, a_lds);
  in.add_operand(b_codes, b_alpha, b_scale, n, k, block, b_ld, b_lds);
  const Range o = range_of(out, groups * m * n * (f32 ? 4 : 2));
  if (in.meets(o) || overlap(o, range_of(offsets, ((int64_t)groups + 1) * 8))) return TFP8_E_ARG;
  ProductArgs p{};
  p.a = Operand{a_codes, a_alpha, a_scale, a_ld, a_lds, 0, 0};
  p.b = Operand{b_codes, b_alpha, b_scale, b_ld, b_lds, 0, 0};
  p.m = m;
  p.n = n;
  p.steps = k / kStep;
  p.shift = log2_of(block);
  p.offsets = offsets;
  p.groups = groups;
  p.rows = rows;
  p.out = out;
  p.ldc = n;
  p.next_c = m * n;
  return launch_product<kGroupedDepth>(p, f32, (hipStream_t)stream);
}

}  // extern "C"
