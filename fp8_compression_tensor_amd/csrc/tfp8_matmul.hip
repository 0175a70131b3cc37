// tfp8_matmul.hip - gfx950 products of compressed operands: C = A^ B^T where A^ and B^ are what
// the codes of A[M, K] and B[N, K] stand for, dense, grouped by rows, and grouped along the
// contraction.
//
// Mathematics.  Both operands are compressed in blocks along K with the same rotation, so a
// block of a row is a^ = H u_a / sqrt(B), u_a = r_a dec(q_a), r_a = s_a / alpha_a (without the
// rotation a^ = u_a).  H / sqrt(B) is orthogonal: a^ . b^ = u_a . u_b, and
//   C[m][n] = sum over blocks of r_a[m] r_b[n] sum_k dec(qa[m][k]) dec(qb[n][k]).
// The inner sum is what the matrix cores compute on the codes as they are; no Hadamard, no
// decompressed copy.  Each 128-deep partial tile is scaled by r_a r_b and added in float32 (float64
// where r_a r_b may leave its range).
#include <math.h>
#include <stdint.h>

#include "../../include/tfp8.h"
#include "tfp8_device.hpp"
#include "tfp8_groups.hpp"
#include "tfp8_host.hpp"

namespace tfp8 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(3))) void lds_const;

constexpr int kStep = 128;  // contraction depth of one matrix instruction

// A compressed operand: rows of codes `ld` bytes apart, rows of scales `lds` floats apart.
struct Operand {
  const uint8_t *codes;
  const float *alpha, *scale;
  int32_t ld, lds;
};

enum : int { kDense = 0, kGroupedRows = 1, kGroupedDepth = 2 };

// Kept small: a launch copies it (16 bytes of arguments take 2.6 us to launch, 208 take 3.5).
struct ProductArgs {
  Operand a, b;            // kGroupedRows: one b after the other
  const int64_t *offsets;
  void *out;               // kGroupedDepth: one [m][n] after the other
  int64_t ldc;
  int32_t m, n;            // rows of A (all groups together, kGroupedRows) and of B
  int32_t rows, groups;    // rows: of the uncompressed operands (kGroupedDepth)
  int32_t steps;           // kStep-deep steps along a row
  int32_t shift;           // log2(block / kStep): so many steps share a scale
  int32_t mtiles, ntiles;
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

// part[j] = x[j] y for all j: the wide form goes over the quarters outermost, so that neighbouring
// instructions do not wait for one another.
template <int N>
__device__ __forceinline__ void mfma_row(f32x4 (&part)[N], const Fragment<true> (&x)[N],
                                         const Fragment<true> &y) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
      part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j].v[t], y.v[t], t ? part[j] : zero, 0, 0,
                                                        0);
    }
}
template <int N>
__device__ __forceinline__ void mfma_row(f32x4 (&part)[N], const Fragment<false> (&x)[N],
                                         const Fragment<false> &y) {
#pragma unroll
  for (int j = 0; j < N; ++j) part[j] = mfma_codes(x[j], y);
}

// A raw buffer descriptor: reads at or past `bytes` give zeros.
__device__ __forceinline__ i32x4 buffer_of(const void *base, int bytes) {
  const uint64_t p = (uint64_t)base;
  return i32x4{__builtin_amdgcn_readfirstlane((int)p),
               __builtin_amdgcn_readfirstlane((int)(p >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

__device__ __forceinline__ const uint8_t *base_of(i32x4 buffer) {
  return (const uint8_t *)((uint64_t)(uint32_t)buffer[0] | (uint64_t)(uint32_t)buffer[1] << 32);
}

// 16 bytes a lane from the buffer at offset voff + soff to LDS, lane l's at to + 16 l.  Written as
// asm because the compiler waits for every such load in flight before any read of LDS, also of
// the other stage; it returns no register, and the caller waits for it with wait_loads().  m0, which
// holds the address, has no other use in these kernels.
__device__ __forceinline__ void load_to_lds(i32x4 buffer, int voff, int soff, const void *to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_const *)to);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(at), "v"(voff), "s"(buffer), "s"(soff)
      : "memory");
}
// Every load of this wavefront, to registers or to LDS, has arrived.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Every LDS access of this wavefront is done,
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// and those of the whole workgroup.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Vectors that may start at any element (global memory takes them at any address).
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16);
}

// Four neighbouring values of a row, of which the first `valid` are inside.
template <bool F32OUT>
__device__ __forceinline__ void store_values(void *out, int64_t at, const f32x4 v, int valid) {
  if constexpr (F32OUT) {
    float *o = (float *)out + at;
    if (valid >= 4) {
      *(f32x4u *)o = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < valid) o[i] = v[i];
    }
  } else {
    __bf16 *o = (__bf16 *)out + at;
    if (valid >= 4) {
      *(u32x2_any *)o = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < valid) o[i] = (__bf16)v[i];
    }
  }
}

// A row of two neighbouring 16 x 16 tiles in bfloat16.  The lanes q = 0..3 of a row hold columns 4 q
// on of each tile (8 bytes); two swaps between lanes 32 and 16 apart give lane q columns 8 q on of
// the 32, so that the four store 64 bytes together.  (4096 x 4096 x 1024: 25.8 us, against
// 29.4 in pieces of 8 bytes.)
__device__ __forceinline__ void store_pair(void *out, int64_t at, int q, f32x4 a, f32x4 b,
                                           int valid) {
  uint32_t x[2] = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
  uint32_t y[2] = {pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(x[i], y[i], false, false);
    const auto u = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
    x[i] = u[0];
    y[i] = u[1];
  }
  __bf16 *o = (__bf16 *)out + at + 8 * q;
  valid -= 8 * q;
  const uint32_t d[4] = {x[0], x[1], y[0], y[1]};
  if (valid >= 8) {
    *(u32x4_any *)o = u32x4{d[0], d[1], d[2], d[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < valid) ((uint16_t *)o)[i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
  }
}

// What a workgroup computes: rows [m0, m0 + mv) of A by rows [n0, n0 + nv) of B over the steps
// [s0, s1), and where it goes.
struct Job {
  const uint8_t *ac, *bc;          // codes of the first rows
  const float *aa, *as, *ba, *bs;  // their scales
  char *out;                       // the first element
  int mv, nv;
  int s0, s1;
};

// The workgroup's tile.  Neighbouring workgroups go to different XCDs, each with an L2 of its own,
// so tiles are dealt out in eight contiguous parts, and run down bands of kBand tiles of A: what an
// XCD works on at one time then shares rows on both sides.  (8192 x 8192 x 8192: 595 us, against
// 677 in the same bands without the parts; one band of 16, 618.)  The parts of a product over
// ragged depths would be uneven (561 us against 454), and stay in plain order.
constexpr int kBand = 4;

// This workgroup's place among `all` tiles (at most one a workgroup); all: it has none.
__device__ __forceinline__ uint32_t place_of_workgroup(uint32_t all) {
  const uint32_t per = all >> 3, over = all & 7, x = blockIdx.x & 7, i = blockIdx.x >> 3;
  return i < per + (x < over) ? x * per + (x < over ? x : over) + i : all;
}

// Row and column of tiles of place `at` in mtiles rows of ntiles.
__device__ __forceinline__ void tile_at(uint32_t at, int mtiles, int ntiles, int &mt, int &nt) {
  const uint32_t band = kBand * (uint32_t)ntiles, in_band = at % band;
  const int b0 = (int)(at / band) * kBand;
  const uint32_t high = mtiles - b0 < kBand ? mtiles - b0 : kBand;
  mt = b0 + (int)(in_band % high);
  nt = (int)(in_band / high);
}

template <int BM, int BN, int MODE, int ES>
__device__ __forceinline__ bool find_job(const ProductArgs &p, Job &t) {
  char *out = (char *)p.out;
  int64_t s0 = 0, s1 = p.steps, m0, bskip = 0, bskip_s = 0;
  int mt = 0, nt = 0;
  if constexpr (MODE == kGroupedRows) {
    // the launch is for the most tiles that groups of any sizes come to; the parts are of those
    // that there are (3200 rows in 16 groups by 2560 x 2048: 43 us, against 83 in parts of the launch,
    // which left the last XCD without work)
    const GroupTile g =
        tile_of_groups(p.offsets, p.groups, p.m, BM, true, [&](int64_t there) -> int64_t {
          const uint32_t all = (uint32_t)there * p.ntiles, at = place_of_workgroup(all);
          if (at >= all) return there;
          tile_at(at, (int)there, p.ntiles, mt, nt);
          return mt;
        });
    if (g.rows <= 0) return false;
    m0 = g.row0;
    t.mv = g.rows;
    if (g.group < 0) {  // rows of no group: zeros
      s1 = 0;
    } else {
      bskip = (int64_t)g.group * p.n * p.b.ld;
      bskip_s = (int64_t)g.group * p.n * p.b.lds;
    }
  } else {
    uint32_t at = blockIdx.x;
    if constexpr (MODE == kGroupedDepth) {
      const uint32_t per = (uint32_t)p.mtiles * p.ntiles, e = at / per;
      at -= e * per;
      const GroupSpan g = span_of_group(p.offsets, p.groups, p.rows, kStep << p.shift, (int)e);
      s0 = g.unit0 << p.shift;
      s1 = (g.unit0 + g.units) << p.shift;
      s1 = s1 < p.steps ? s1 : p.steps;
      s0 = s0 < s1 ? s0 : s1;
      out += (int64_t)e * p.m * p.n * ES;
    } else {
      at = place_of_workgroup(gridDim.x);
    }
    tile_at(at, p.mtiles, p.ntiles, mt, nt);
    m0 = (int64_t)mt * BM;
    t.mv = (int)(p.m - m0 < BM ? p.m - m0 : BM);
  }
  const int64_t n0 = (int64_t)nt * BN;
  t.nv = (int)(p.n - n0 < BN ? p.n - n0 : BN);
  t.s0 = (int)s0;
  t.s1 = (int)s1;
  t.ac = p.a.codes + m0 * p.a.ld;
  t.aa = p.a.alpha + m0 * p.a.lds;
  t.as = p.a.scale + m0 * p.a.lds;
  t.bc = p.b.codes + bskip + n0 * p.b.ld;
  t.ba = p.b.alpha + bskip_s + n0 * p.b.lds;
  t.bs = p.b.scale + bskip_s + n0 * p.b.lds;
  t.out = out + (m0 * p.ldc + n0) * ES;
  return true;
}

// Which ranges the factors r = s / alpha of an operand come from.  r_a r_b is one float32 factor of a
// block's sum.  An r below float32's normal range (blocks of values below about 2^-115) has lost
// bits, which is below 2^-123 of a result for each kStep codes as long as the other operand's r is
// at most 1.  A tile where an r of one operand may be so small (alpha above 2^84: every r below 2^-126
// has one, whatever its target) and one of the other above 1 is computed again by wide_range_tile; so
// is one where both have an r above 2^31 (no r reaches 2^96), whose product may be infinite and make NaN
// of a sum that is 0.
enum : int { kTinyA = 1, kLargeA = 2, kHugeA = 4, kTinyB = 8, kLargeB = 16, kHugeB = 32 };

// Notes four blocks of a row of each lane, the rows all of A or all of B; as integers, which order like
// these positive floats.  Noting and asking at the end take 1% of a large product, 0.2 us of one of
// few rows.
__device__ __forceinline__ void note_range(const f32x4 s, const f32x4 alpha, bool is_a, int &saw) {
  int a[4], most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_int(alpha[i]);
    most = max(most, __float_as_int(s[i]));
  }
  const int least = min(min(a[0], a[1]), min(a[2], a[3]));
  const uint64_t tiny = __ballot(max(max(a[0], a[1]), max(a[2], a[3])) > __float_as_int(0x1p84f));
  const uint64_t large = __ballot(most > least);
  if (__builtin_expect((tiny | large) != 0, 0)) {
    const uint64_t huge = __ballot(__int_as_float(most) > 0x1p31f * __int_as_float(least));
    const int seen = (tiny ? kTinyA : 0) | (large ? kLargeA : 0) | (huge ? kHugeA : 0);
    saw |= is_a ? seen : seen * (kTinyB / kTinyA);
  }
}

// A wavefront's `saw` to its word of LDS, and, after a barrier, a wavefront's word to each lane and
// whether together they ask for wide_range_tile.
__device__ __forceinline__ void tell(float *words, int w, int saw) { words[w] = __int_as_float(saw); }
template <int WAVES>
__device__ __forceinline__ int told(const float *words) {
  return __float_as_int(words[threadIdx.x & (WAVES - 1)]);
}
__device__ __forceinline__ bool wide_range(int word) {
  if (__builtin_expect(__ballot(word) == 0, 1)) return false;
  return (__ballot(word & kTinyA) && __ballot(word & kLargeB)) ||
         (__ballot(word & kTinyB) && __ballot(word & kLargeA)) ||
         (__ballot(word & kHugeA) && __ballot(word & kHugeB));
}

// LDS of a tile: two stages of a step's codes, A's rows then B's (four measured no
// faster, and halve what fits), and scales r: those of a step for each stage, or (CHUNK > 0) those of
// CHUNK blocks.  KS > 1: the workgroup's wavefronts form KS teams with stages of their own, and team
// g takes steps g, g + KS, ...
template <int BM_, int BN_, int KS_, int CHUNK_>
struct Stages {
  static constexpr int BM = BM_, BN = BN_, KS = KS_, CHUNK = CHUNK_;
  static_assert(KS == 1 || CHUNK > 0, "teams share the scales of a chunk");
  alignas(1024) uint8_t codes[KS][2][(BM + BN) * kStep];
  float r[CHUNK ? CHUNK : 2][BM + BN];
};

// Filling the stages of one team of NW wavefronts.
template <class STAGES, int NW>
struct Feed {
  static constexpr int BM = STAGES::BM, BN = STAGES::BN, CHUNK = STAGES::CHUNK;
  static constexpr int ROWS = BM + BN, NT = 64 * NW;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // a wavefront's loads a step
  static constexpr int SC = (ROWS + NT - 1) / NT;           // rows whose scales a thread prepares
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole loads of one operand");
  static_assert(BM % 64 == 0 && ROWS % 64 == 0, "a wavefront's scales are of one operand");

  STAGES &lds;
  int team, w, shift, first, blocks;  // w: the wavefront within its team
  int saw = 0;                        // of note_range
  i32x4 ra[LA], rb[LB];
  int va, vb;
  const char *sp[SC], *ap[SC];  // a wavefront's rows are of one operand
  uint32_t at0[SC];
  f32x4 sv[SC], av[SC];

  // A wavefront's load instruction fills 8 rows of 128 bytes of LDS, lane i the i-th 16 bytes; it
  // takes them from chunk (i & 7) ^ (row & 7) of its row, so that the lanes that read a column of
  // fragments touch all banks.  Each instruction has a descriptor of its own, from its first row on
  // to the operand's end, past which rows read as zeros.
  __device__ __forceinline__ Feed(STAGES &l, const ProductArgs &p, const Job &t)
      : lds(l), shift(p.shift) {
    const int lane = threadIdx.x & 63;
    team = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / NW;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW;
    const int tid = w * 64 + lane;
    const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    va = (lane >> 3) * (int)p.a.ld + chunk;
    vb = (lane >> 3) * (int)p.b.ld + chunk;
    const int k = (int)p.steps * kStep, lda = (int)p.a.ld, ldb = (int)p.b.ld;  // products < 2^31
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int row = (i * NW + w) * 8, left = (t.mv - 1 - row) * lda + k;
      ra[i] = buffer_of(t.ac + row * lda, left > 0 ? left : 0);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int row = (i * NW + w) * 8, left = (t.nv - 1 - row) * ldb + k;
      rb[i] = buffer_of(t.bc + row * ldb, left > 0 ? left : 0);
    }
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const bool isa = w * 64 + i * NT < BM;
      int rr = tid + i * NT - (isa ? 0 : BM);
      const int last = (isa ? t.mv : t.nv) - 1;
      rr = rr < last ? rr : last;
      at0[i] = (uint32_t)(rr * (int)(isa ? p.a.lds : p.b.lds)) * 4;  // below 2^30
      sp[i] = (const char *)(isa ? t.as : t.bs);
      ap[i] = (const char *)(isa ? t.aa : t.ba);
    }
    first = t.s0 >> shift;
    blocks = (int)(p.steps >> shift);
  }

  // The part-th of `parts` shares of a step's loads.
  __device__ __forceinline__ void load_step(int s, int stage, int part = 0, int parts = 1) {
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) {
      if (i * parts / (LA + LB) != part) continue;
      if (i < LA)
        load_to_lds(ra[i], va, s * kStep, &lds.codes[team][stage][(i * NW + w) * 1024]);
      else
        load_to_lds(rb[i - LA], vb, s * kStep,
                    &lds.codes[team][stage][BM * kStep + ((i - LA) * NW + w) * 1024]);
    }
  }
  // Scales, r = scale / alpha of every row (A's, then B's).
  //
  // CHUNK > 0: the next CHUNK blocks' at once, from block b on, four to a thread.
  __device__ __forceinline__ void fill_scales(int b, const ProductArgs &p, const Job &t) {
    constexpr int QUADS = CHUNK / 4, ALL = NT * STAGES::KS, EACH = ROWS * QUADS / ALL;
    static_assert(CHUNK % 4 == 0 && ROWS * QUADS % ALL == 0, "whole quads for every thread");
    f32x4 x[EACH], y[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = (int)threadIdx.x + i * ALL, row = at / QUADS, k = b + at % QUADS * 4;
      const bool isa = row < BM;
      int rr = isa ? row : row - BM;
      const int last = (isa ? t.mv : t.nv) - 1;
      rr = rr < last ? rr : last;
      const int64_t from = (int64_t)rr * (isa ? p.a.lds : p.b.lds) + k;
      const float *ss = (isa ? t.as : t.bs) + from, *aa = (isa ? t.aa : t.ba) + from;
      x[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      y[i] = f32x4{1.0f, 1.0f, 1.0f, 1.0f};
      if (k + 4 <= blocks) {
        x[i] = *(const f32x4u *)ss;
        y[i] = *(const f32x4u *)aa;
      } else {
#pragma unroll
        for (int u = 0; u < 3; ++u)
          if (k + u < blocks) {
            x[i][u] = ss[u];
            y[i][u] = aa[u];
          }
      }
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = (int)threadIdx.x + i * ALL, row = at / QUADS, k = at % QUADS * 4;
      note_range(x[i], y[i], (i * ALL + (team * NW + w) * 64) / QUADS < BM, saw);
#pragma unroll
      for (int u = 0; u < 4; ++u) lds.r[k + u][row] = x[i][u] * __builtin_amdgcn_rcpf(y[i][u]);
    }
  }
  // CHUNK = 0: thread t prepares row t's.  Rows' lie a row apart in memory, a cache line each, so
  // four blocks' are loaded at once: called for every step, this loads at the first of four
  // blocks.  (Laid out [block][row] by a launch before this one, they cost less here: 539 us against
  // 555 at 8192 x 8192 x 8192, but with that launch 80 against 73 at 4096 x 4096 x 4096.)
  __device__ __forceinline__ void load_scales(int s) {
    if constexpr (CHUNK > 0) return;
    const int at = s >> shift;
    if (((at - first) & 3) || (s & ((1 << shift) - 1))) return;
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const char *ss = sp[i] + at * 4, *aa = ap[i] + at * 4;
      if (at + 4 <= blocks) {
        sv[i] = *(const f32x4u *)(ss + at0[i]);
        av[i] = *(const f32x4u *)(aa + at0[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sv[i][k] = at + k < blocks ? *(const float *)(ss + at0[i] + 4 * k) : 0.0f;
          av[i][k] = at + k < blocks ? *(const float *)(aa + at0[i] + 4 * k) : 1.0f;
        }
      }
    }
  }
  __device__ __forceinline__ void put_scales(int s, int stage) {
    if constexpr (CHUNK > 0) return;
    const int k = ((s >> shift) - first) & 3;
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      if (k == 0) note_range(sv[i], av[i], w * 64 + i * NT < BM, saw);
      const float x = k & 2 ? (k & 1 ? sv[i][3] : sv[i][2]) : (k & 1 ? sv[i][1] : sv[i][0]);
      const float y = k & 2 ? (k & 1 ? av[i][3] : av[i][2]) : (k & 1 ? av[i][1] : av[i][0]);
      const int row = (int)threadIdx.x + i * NT;
      if (ROWS % NT == 0 || row < ROWS) lds.r[stage][row] = x * __builtin_amdgcn_rcpf(y);
    }
  }
};

// Lane l takes chunks q and q + 4 of row l & 15 of a 16-row tile; `at` is fragment_offset of the
// tile's first row.  With these chunks a read takes 4 cycles, all banks busy (measured; 2 q and
// 2 q + 1, which look as good, meet in pairs and take 8).
__device__ __forceinline__ int fragment_offset(int row, int q, int l16) {
  return (row + l16) * kStep + ((q ^ (l16 & 7)) << 4);
}
template <bool WIDE>
__device__ __forceinline__ Fragment<WIDE> read_fragment(const uint8_t *codes, int at) {
  return make_fragment<WIDE>(*(const u32x4 *)(codes + at), *(const u32x4 *)(codes + (at ^ 64)));
}

// The loop over steps, for wavefronts of TM x TN tiles.  The scaled addition of a tile's partial
// products follows TN matrix instructions behind the one that makes them, so that neither waits for
// the other.  One barrier a step, before the last row of tiles: by then the step's fragments are in
// registers, so the loads of the step two ahead may overwrite them, and the next step's first
// fragments are read under the last row's products.
template <int TM, int TN, bool WIDE, class STAGES, class FEED>
__device__ __forceinline__ void run_steps(STAGES &lds, FEED &feed, const ProductArgs &p,
                                          const Job &job, int mrow, int nrow,
                                          f32x4 (&acc)[TM][TN]) {
  constexpr int KS = STAGES::KS, BM = STAGES::BM, CHUNK = STAGES::CHUNK;
  constexpr int NP = TM >= 8 ? 3 : TM >= 3 ? 2 : 1;  // a step's loads go out in this many shares
  static_assert(CHUNK > 0 || NP > 1, "a step's scales are loaded with its last share");
  const int s0 = job.s0, s1 = job.s1;
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int fa0 = fragment_offset(mrow, q, l16), fb0 = fragment_offset(BM + nrow, q, l16);
  const int team = KS > 1 ? feed.team : 0;
  const auto &codes = lds.codes[team];
  int s = s0 + team;
  int chunk0 = s0 >> p.shift;  // first block of the scales in LDS (CHUNK)
  // With teams every step issues its loads, past the end those of the last step again, so that a
  // team that is a step short works on codes (with its scales taken as zero).
  const auto load = [&](int x, int slot, int part, int parts) {
    if (KS > 1)
      feed.load_step(x < s1 ? x : s1 - 1, slot, part, parts);
    else if (x < s1)
      feed.load_step(x, slot, part, parts);
  };
  feed.load_scales(s);
  load(s, 0, 0, 1);
  wait_loads();
  feed.put_scales(s, 0);
  if constexpr (CHUNK > 0) feed.fill_scales(chunk0, p, job);
  lds_barrier();
  load(s + KS, 1, 0, NP);
  // where the scales of step x, in slot y, are
  const auto scales = [&](int x, int y) {
    return CHUNK > 0 ? lds.r[((x < s1 ? x : s1 - 1) >> p.shift) - chunk0] : lds.r[y];
  };
  Fragment<WIDE> fb[TN], fa;
  f32x4 rb[TN], part[TN];
  float ra, rprev = 0.0f;  // A's scales of this row of tiles and of the one before
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    fb[j] = read_fragment<WIDE>(codes[0], fb0 + j * 16 * kStep);
    rb[j] = part[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  fa = read_fragment<WIDE>(codes[0], fa0);
  ra = KS == 1 || s < s1 ? scales(s, 0)[mrow + l16] : 0.0f;
  // part[j] of the row of tiles before, scaled and added
  auto add_part = [&](f32x4 (&to)[TN], int j) {
#pragma unroll
    for (int k = 0; k < 4; ++k) to[j][k] = fmaf(part[j][k], rprev * rb[j][k], to[j][k]);
    // keeps the addition here: the compiler would move it past the branches below, and keep
    // every partial product until then
    asm volatile("" : "+v"(to[j]));
  };
  for (int slot = 0; s - team < s1; s += KS, slot ^= 1) {
    const int ahead = slot ^ 1;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const bool last = i == TM - 1;
      if (last) {
        wait_loads();
        if (s + 1 < s1) feed.put_scales(s + 1, ahead);
        lds_barrier();
        load(s + 2 * KS, slot, 0, NP);
        if constexpr (CHUNK > 0) {
          const int n0 = s - team + KS, n1 = n0 + KS - 1;  // the teams' next steps
          if (n0 < s1 && (n1 >> p.shift) - chunk0 >= CHUNK) {
            chunk0 = n0 >> p.shift;
            feed.fill_scales(chunk0, p, job);
            lds_barrier();
          }
        }
      } else if (i + 1 < NP) {
        load(s + KS, ahead, i + 1, NP);
        if (i + 2 == NP && s + 1 < s1) feed.load_scales(s + 1);
      }
      const int ns = last ? ahead : slot;
      const int ni = last ? 0 : i + 1;
      const Fragment<WIDE> fn = read_fragment<WIDE>(codes[ns], fa0 + ni * 16 * kStep);
      const int sn = last ? s + KS : s;
      const float rn = KS == 1 || sn < s1 ? scales(sn, ns)[mrow + ni * 16 + l16] : 0.0f;
      // B's scales of this step replace the last one's once its last row is added
      auto next_scales = [&](int j) {
        if (i == 0) rb[j] = *(const f32x4 *)&scales(s, slot)[BM + nrow + j * 16 + 4 * q];
      };
      if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          add_part(acc[i ? i - 1 : TM - 1], j);
          next_scales(j);
        }
        mfma_row(part, fb, fa);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (last) fb[j] = read_fragment<WIDE>(codes[ns], fb0 + j * 16 * kStep);
      } else {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          add_part(acc[i ? i - 1 : TM - 1], j);
          next_scales(j);
          part[j] = mfma_codes(fb[j], fa);
          if (last) fb[j] = read_fragment<WIDE>(codes[ns], fb0 + j * 16 * kStep);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      fa = fn;
      rprev = ra;
      ra = rn;
    }
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) add_part(acc[TM - 1], j);
  if (KS > 1) wait_loads();  // no load may arrive after the workgroup has given its LDS back
}

// A tile once more, where the product of two r need not be a float32 (note_range): the factors and
// the sums over steps in float64.  A wavefront takes one tile of 16 x 16 after the other, its codes
// and scales straight from memory, rows past the end those of the last row again.  The kernel's
// arguments are read again, so that no registers keep them through the loops for this.  4096 x 4096 x
// 4096 takes 1.5 ms where every tile comes to this, 64 x 5120 x 5120 55 us.
template <bool F32OUT, int WAVES>
__device__ __forceinline__ void wide_range_tile(const Job &t) {
  auto *args = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(args));
  ProductArgs p;
  __builtin_memcpy(&p, (const void *)args, sizeof p);
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int across = (t.nv + 15) / 16, tiles = (t.mv + 15) / 16 * across;
  const auto load = [&](const uint8_t *codes) {
    const u32x4 lo = *(const u32x4 *)(codes + 16 * q), hi = *(const u32x4 *)(codes + 16 * q + 64);
    return make_fragment<F32OUT>(lo, hi);
  };
  const auto factor = [](const float *scale, const float *alpha, int at) {
    return (double)scale[at] * (double)__builtin_amdgcn_rcpf(alpha[at]);
  };
  for (int at = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); at < tiles; at += WAVES) {
    const int row = at / across * 16 + l16, c0 = at % across * 16, col = c0 + 4 * q;
    const int r = row < t.mv ? row : t.mv - 1;
    const int c = c0 + l16 < t.nv ? c0 + l16 : t.nv - 1;
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    for (int s = t.s0; s < t.s1; ++s) {
      const Fragment<F32OUT> fa = load(t.ac + r * p.a.ld + s * kStep);  // offsets below 2^31
      const Fragment<F32OUT> fb[1] = {load(t.bc + c * p.b.ld + s * kStep)};
      f32x4 part[1];
      mfma_row(part, fb, fa);
      const int b = s >> p.shift;
      const double ra = factor(t.as, t.aa, r * p.a.lds + b);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int ck = col + k < t.nv ? col + k : t.nv - 1;
        sum[k] += (double)part[0][k] * (ra * factor(t.bs, t.ba, ck * p.b.lds + b));
      }
    }
    const f32x4 v = {(float)sum[0], (float)sum[1], (float)sum[2], (float)sum[3]};
    if (row < t.mv) store_values<F32OUT>(t.out, row * p.ldc + col, v, t.nv - col);
  }
}

// One tile of BM x BN by WM x WN wavefronts (of KS teams).
//
// What bounds it.  bfloat16, tiles of 256 x 256: 8192 x 16384 x 4096 in blocks of 256 takes 560 to
// 645 us on different cards, 1.7 to 1.96 PFLOP/s (a library product of 8-bit operands with one scale
// each reaches 3.1), some 4600 cycles a step, at a clock that the power limit holds near 1.9 GHz.  No one unit
// is full: the matrix units are busy 44% of the cycles (2048 a step), half of that beside vector
// instructions; vector instructions, eight of them with each matrix instruction for its scaled addition, take
// 59% of a SIMD's issue and scalar ones 16%; and a wavefront waits 26% of its time for loads, LDS or the
// barrier, and 28% for its turn to issue.  Two wavefronts a SIMD, in step at the barrier, leave gaps
// that neither fills.  Codes that are all zero take 13% less time at the same work, and a loop over
// tiles that fetches the next one's codes under the stores of this one gained nothing.  16384 rows in
// 8 groups by 5120 x 4096: 435 to 484 us, the same rate less its last round of tiles, a third
// full; the weight gradient of 16384 rows in 8 groups, 4096 x 2560 each, 230 us, 1.49 PFLOP/s.
// float32, tiles of 128 x 128 by four wavefronts, two workgroups a compute unit: widening the codes
// takes eight more vector instructions for each 16 x 16 tile and step, each code being widened by both
// wavefronts that use it, and the matrix instructions have half the rate.  8192 x 8192 x 8192: 1040 to
// 1120 us, about 1.02 PFLOP/s.  8 groups of 16384 rows in all, 4096 x 2560 each: 403 to 465 us, 0.74
// to 0.85 PFLOP/s; a tile is 16 steps deep there.  (In tiles of 256 x 128 by eight wavefronts 1093 us,
// and 428 where this takes 420; 6400 rows in 16 groups by 5120 x 1024 152 us, against 109.)  In tiles
// of 64 x 64 (1003 x 2571 x 2560: 25 to 29 us) widening is 64 of a wavefront's 104 vector instructions
// a step, for four 16 x 16 tiles, again twice for each code; they fill somewhat over half of the issue
// while a compute unit has a workgroup, which, with 2.6 tiles for each, is some 70% of the time.
// Larger tiles, which widen less, leave compute units without one.
//
// The kernel only calls this function: a kernel's own body is also read by the host's pass, which
// does not know these builtins.
template <int BM, int BN, int WM, int WN, int KS, int CHUNK, int MODE, bool F32OUT>
__device__ __forceinline__ void matmul_tile(const ProductArgs &p) {
  constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN, KEEP = TM / KS;
  using STAGES = Stages<BM, BN, KS, CHUNK>;
  __shared__ STAGES lds;
  Job t;
  if (!find_job<BM, BN, MODE, F32OUT ? 4 : 2>(p, t)) return;
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = all % (WM * WN), team = all / (WM * WN);
  const int mrow = w / WN * TM * 16, nrow = w % WN * TN * 16;
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (t.s0 < t.s1) {
    Feed<STAGES, WM * WN> feed(lds, p, t);
    run_steps<TM, TN, F32OUT>(lds, feed, p, t, mrow, nrow, acc);
    // what other wavefronts still read of the scales is of a step past the end, and not used
    tell(&lds.r[0][0], all, feed.saw);
    lds_barrier();
    if (__builtin_expect(wide_range(told<WM * WN * KS>(&lds.r[0][0])), 0))
      return wide_range_tile<F32OUT, WM * WN * KS>(t);
  }
  // row of tiles i of this wavefront
  const auto store_row = [&](int i, const f32x4 (&v)[TN]) {
    const int row = mrow + i * 16 + l16;
    if constexpr (F32OUT) {
      if (row < t.mv) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int col = nrow + j * 16 + 4 * q;
          store_values<true>(t.out, row * p.ldc + col, v[j], t.nv - col);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; j += 2) {  // every lane takes part in the swaps
        const int col = nrow + j * 16;
        store_pair(t.out, row * p.ldc + col, q, v[j], v[j + 1], row < t.mv ? t.nv - col : 0);
      }
    }
  };
  if constexpr (KS == 1) {
#pragma unroll
    for (int i = 0; i < TM; ++i) store_row(i, acc[i]);
  } else {
    // two teams: each stores half of its rows of tiles, and gives the other half to its counterpart
    static_assert(KS == 2 && sizeof(lds.codes) >= 2 * WM * WN * KEEP * TN * 1024, "teams' sums");
    f32x4 *sum = (f32x4 *)&lds.codes[0][0][0] + lane;
    const auto at = [&](int to, int i, int j) {
      return (((to * WM * WN + w) * KEEP + i) * TN + j) * 64;
    };
    lds_barrier();  // both teams' loads have arrived, and their fragments are in registers
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        sum[at(team ^ 1, i, j)] = team == 0 ? acc[i + KEEP][j] : acc[i][j];
    lds_barrier();
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      f32x4 v[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const f32x4 o = sum[at(team, i, j)];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[j][k] = (team == 0 ? acc[i][j][k] : acc[i + KEEP][j][k]) + o[k];
      }
      store_row(team * KEEP + i, v);
    }
  }
}

template <int BM, int BN, int WM, int WN, int KS, int CHUNK, int MODE, bool F32OUT>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void k_matmul_tile(ProductArgs p) {
  matmul_tile<BM, BN, WM, WN, KS, CHUNK, MODE, F32OUT>(p);
}

// --------------------------------------------------------------------------------------------
// Few rows (decoding): B's bytes bound the product.  A workgroup takes one tile of 16 MT rows of A
// (its group's) by 16 TN of B, and its eight wavefronts divide the depth: each computes the whole tile
// over its share of the steps, and the eight are added up through LDS in a fixed order at the end.
// Each wavefront has a stage of LDS to itself, so there is no barrier in the loop: it waits for
// its own loads alone, reads a step's codes into registers, and sends the next step's loads out before
// it multiplies.  (Fragments loaded straight from memory, 16 rows of 64 bytes an
// instruction in the order of the lanes, come at 9.6 TB/s over the chip, from the L1 cache too; whole
// lines through LDS come at 28.)
//
// 24 x 10240 x 5120: 14.1 us, 4.0 TB/s, in 32 x 48 tiles (14.5 in 32 x 64, 19 in 32 x 32, whose 320
// workgroups are more than one round); 48 rows in 16 groups, 2560 x 4096 each: 36 us, 4.7 TB/s.  (The
// compress kernel streams 6.1 TB/s from HBM; of three operands read in turn here a part stays in the 256 MB
// cache.)  One row of 4096 x 4096, 2.9 TB/s, takes 6.2 us, of which its bytes are 2.9 and the start,
// the first loads' latency and the sum over the wavefronts the rest.  Scales are prepared in LDS,
// kSplitBlocks blocks at a time.
constexpr int kSplitWaves = 8, kSplitBlocks = 64;

// 32 codes of a lane, as stored.
struct Codes {
  u32x4 lo, hi;
};
__device__ __forceinline__ Codes read_codes(const uint8_t *codes, int at) {
  return Codes{*(const u32x4 *)(codes + at), *(const u32x4 *)(codes + (at ^ 64))};
}

template <int MT, int TN, int MODE, bool F32OUT>
__device__ __forceinline__ void matmul_split(const ProductArgs &p) {
  constexpr int BM = 16 * MT, BN = 16 * TN, ROWS = BM + BN, NT = 64 * kSplitWaves;
  constexpr int QUADS = kSplitBlocks / 4, EACH = (ROWS * QUADS + NT - 1) / NT;
  constexpr int LOADS = ROWS / 8;  // a step's
  __shared__ struct {
    union {
      alignas(1024) uint8_t codes[kSplitWaves][ROWS * kStep];
      f32x4 sum[kSplitWaves][MT * TN][64];
    };
    float r[kSplitBlocks][ROWS];
  } lds;
  Job t;
  if (!find_job<BM, BN, MODE, F32OUT ? 4 : 2>(p, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  // loads: 8 rows each, as in Feed
  i32x4 from[LOADS];
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  const int va = (lane >> 3) * (int)p.a.ld + chunk, vb = (lane >> 3) * (int)p.b.ld + chunk;
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const bool isa = i < BM / 8;
    const int row = isa ? i * 8 : i * 8 - BM;
    const int ld = (int)(isa ? p.a.ld : p.b.ld);  // below 2^22, and at most 64 rows
    const int left = ((isa ? t.mv : t.nv) - 1 - row) * ld + (int)p.steps * kStep;
    from[i] = buffer_of((isa ? t.ac : t.bc) + row * ld, left > 0 ? left : 0);
  }
  const auto load = [&](int s) {  // past the end: the last step again, which is left out
    const int k0 = (s < t.s1 ? s : t.s1 - 1) * kStep;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_to_lds(from[i], i < BM / 8 ? va : vb, k0, &lds.codes[w][i * 1024]);
  };
  const int fa0 = fragment_offset(0, q, l16), fb0 = fragment_offset(BM, q, l16);
  Codes ca[MT], cb[TN];
  const auto read = [&] {
#pragma unroll
    for (int j = 0; j < TN; ++j) cb[j] = read_codes(lds.codes[w], fb0 + j * 16 * kStep);
#pragma unroll
    for (int i = 0; i < MT; ++i) ca[i] = read_codes(lds.codes[w], fa0 + i * 16 * kStep);
  };
  f32x4 acc[MT][TN];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int blocks = (int)(p.steps >> p.shift);
  int saw = 0;  // of note_range

  for (int c0 = t.s0; c0 < t.s1; c0 += kSplitBlocks << p.shift) {
    // this wavefront's share of the steps whose scales fit
    const int c1 = c0 + (kSplitBlocks << p.shift) < t.s1 ? c0 + (kSplitBlocks << p.shift) : t.s1;
    const int share = (c1 - c0 + kSplitWaves - 1) / kSplitWaves;
    int s = c0 + w * share;
    const int e = s + share < c1 ? s + share : c1;
    load(s);
    const int b0 = c0 >> p.shift;
    if (c0 != t.s0) __syncthreads();  // the scales before are no longer read
    f32x4 x[EACH], y[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = tid + i * NT, row = at / QUADS, k = b0 + at % QUADS * 4;
      x[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      y[i] = f32x4{1.0f, 1.0f, 1.0f, 1.0f};
      if (ROWS * QUADS % NT == 0 || row < ROWS) {
        const bool isa = row < BM;
        int rr = isa ? row : row - BM;
        const int last = (isa ? t.mv : t.nv) - 1;
        rr = rr < last ? rr : last;
        const int64_t off = (int64_t)rr * (isa ? p.a.lds : p.b.lds) + k;
        const float *ss = (isa ? t.as : t.bs) + off, *aa = (isa ? t.aa : t.ba) + off;
        if (k + 4 <= blocks) {
          x[i] = *(const f32x4u *)ss;
          y[i] = *(const f32x4u *)aa;
        } else {
#pragma unroll
          for (int u = 0; u < 3; ++u)
            if (k + u < blocks) {
              x[i][u] = ss[u];
              y[i][u] = aa[u];
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = tid + i * NT, row = at / QUADS, k = at % QUADS * 4;
      note_range(x[i], y[i], (i * NT + w * 64) / QUADS < BM, saw);
      if (ROWS * QUADS % NT == 0 || row < ROWS)
#pragma unroll
        for (int u = 0; u < 4; ++u) lds.r[k + u][row] = x[i][u] * __builtin_amdgcn_rcpf(y[i][u]);
    }
    __syncthreads();
    const auto multiply = [&](const Codes (&xa)[MT], const Codes (&xb)[TN], int step) {
      const float *r = lds.r[(step >> p.shift) - b0];
      Fragment<F32OUT> fb[TN];
      f32x4 rb[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        fb[j] = make_fragment<F32OUT>(xb[j].lo, xb[j].hi);
        rb[j] = *(const f32x4 *)&r[BM + j * 16 + 4 * q];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const Fragment<F32OUT> fa = make_fragment<F32OUT>(xa[i].lo, xa[i].hi);
        const float ra = r[i * 16 + l16];
        f32x4 part[TN];
        mfma_row(part, fb, fa);
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[i][j][k] = fmaf(part[j][k], ra * rb[j][k], acc[i][j][k]);
      }
    };
    wait_loads();
    read();
    for (; s < e; ++s) {
      Codes xa[MT], xb[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) xb[j] = cb[j];
#pragma unroll
      for (int i = 0; i < MT; ++i) xa[i] = ca[i];
      wait_lds();
      load(s + 1);
      multiply(xa, xb, s);
      wait_loads();
      read();
    }
    wait_lds();
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) lds.sum[w][i * TN + j][lane] = acc[i][j];
  tell(&lds.r[0][0], w, saw);
  __syncthreads();
  static_assert(MT * TN <= kSplitWaves, "a 16 x 16 tile a wavefront");
  const int word = told<kSplitWaves>(&lds.r[0][0]);
  f32x4 v;
  if (w < MT * TN) {
    v = lds.sum[0][w][lane];
#pragma unroll
    for (int k = 1; k < kSplitWaves; ++k) {
      const f32x4 o = lds.sum[k][w][lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += o[c];
    }
  }
  if (__builtin_expect(wide_range(word), 0)) {
    t.ac = base_of(from[0]);  // two pointers fewer to keep through the loop
    t.bc = base_of(from[BM / 8]);
    return wide_range_tile<F32OUT, kSplitWaves>(t);
  }
  if (w < MT * TN) {
    const int row = w / TN * 16 + l16, col = w % TN * 16 + 4 * q;
    if (row < t.mv) store_values<F32OUT>(t.out, row * p.ldc + col, v, t.nv - col);
  }
}

template <int MT, int TN, int MODE, bool F32OUT>
__global__ __launch_bounds__(64 * kSplitWaves, 2) void k_matmul_split(ProductArgs p) {
  matmul_split<MT, TN, MODE, F32OUT>(p);
}

}  // namespace tfp8

namespace {

using namespace tfp8;

bool product_block_ok(int32_t block) { return block == 128 || block == 256 || block == 512; }

// How long a kernel takes for tiles of bm x bn (ns): `first` and `step` a step where every compute
// unit has one workgroup, and the same where it has `slots`, which is counted as a full round.  That many
// are resident together, save for three float32 kernels whose registers let fewer in (64 x 64: three of
// the four counted; with two teams, one of two; 16 x 16: three of four): there a full round is more than
// one of the hardware's, and its time, fitted as it is, holds their sum.  From the times of 475 products
// of each output type, of 1 to 4096 rows and 512 to 16384 columns, 640 to 5120 deep, dense, in 4
// to 32 groups and by groups along the depth, a ninth of them with operands that no cache holds; fitted
// so that the choice below costs least: what it picks takes 0.8% longer than the best of these
// kernels on average for bfloat16 outputs, 1.5% for float32 (a choice by the number of rows alone took
// 20% longer, up to 4 times as long).  Products less than five steps deep lie outside the fit.
// slots = 0: no such kernel.
struct Pace {
  int bm, bn, threads, slots;
  int64_t first, step, first_full, step_full;
};
enum : int { kLarge, kMiddle, kSmall, kSmallTeams, kFew, kFew32, kFew48, kKinds };
constexpr Pace kPace[2][kKinds] = {{{256, 256, 512, 1, 11410, 2320, 11410, 2320},
                                    {128, 128, 512, 2, 3590, 1310, 5590, 1450},
                                    {64, 64, 256, 4, 2330, 460, 4230, 1290},
                                    {64, 64, 512, 2, 3080, 360, 4610, 690},
                                    {16, 16, 512, 4, 3010, 17, 4290, 251},
                                    {32, 32, 512, 2, 3670, 95, 5310, 277},
                                    {32, 48, 512, 1, 3250, 160, 3250, 160}},
                                   {{128, 128, 256, 2, 6570, 1200, 6870, 1780},
                                    {},
                                    {64, 64, 256, 4, 2940, 550, 6420, 1230},
                                    {64, 64, 512, 2, 3560, 470, 8090, 1150},
                                    {16, 16, 512, 4, 3220, 30, 5790, 203},
                                    {32, 32, 512, 2, 3990, 112, 7000, 281},
                                    {32, 48, 512, 1, 3460, 186, 3460, 186}}};

int64_t estimate(const Pace &k, int64_t tiles, int64_t steps, int64_t cus) {
  const int64_t one = k.first + steps * k.step, full = k.first_full + steps * k.step_full;
  const int64_t round = k.slots * cus, rest = tiles % round;
  int64_t t = tiles / round * full;
  if (rest > cus)
    t += one + (full - one) * (rest - cus) / (round - cus);
  else if (rest > 0)
    t += one;
  return t;
}

// The kernel whose rounds of workgroups are done first: large tiles use the matrix cores best, small
// ones leave less over at the edges and in the last round, two teams halve the steps of a product
// with few tiles, and the kernels for few rows divide them by eight.
template <int MODE, bool F32OUT>
tfp8_status launch_product(ProductArgs p, hipStream_t st) {
  const int64_t times = MODE == kGroupedDepth ? p.groups : 1, cus = cu_count();
  const int64_t m = p.m, n = p.n;
  const int64_t steps =
      MODE == kGroupedDepth ? ((int64_t)p.rows / p.groups + kStep - 1) / kStep : p.steps;
  int best = -1;
  int64_t least = 0, grid = 0;
  for (int i = 0; i < (MODE == kGroupedDepth ? kFew : kKinds); ++i) {
    const Pace &k = kPace[F32OUT][i];
    if (k.slots == 0) continue;
    const int64_t nt = (n + k.bn - 1) / k.bn;
    int64_t mt = (m + k.bm - 1) / k.bm, most = mt;
    if (MODE == kGroupedRows) {
      // as a rule a tile for each group, and half of one more on average; at most as many as
      // groups of any sizes come to, with the rows before the first and past the last as two more
      const int64_t some = m < p.groups ? m : p.groups, all = m < p.groups + 2 ? m : p.groups + 2;
      mt = m / k.bm + p.groups / 2;
      mt = mt < some ? some : mt;
      most = (m + all * (k.bm - 1)) / k.bm;
    }
    if (most * nt > (((int64_t)1 << 32) - 1) / k.threads / times) continue;  // HIP's limit
    const int64_t ns = estimate(k, mt * nt * times, steps, cus);
    if (best < 0 || ns < least) {
      best = i;
      least = ns;
      p.mtiles = (int32_t)most;
      p.ntiles = (int32_t)nt;
      grid = most * nt * times;
    }
  }
  if (best < 0) return TFP8_E_SIZE;
  const auto run = [&](void (*kernel)(ProductArgs)) {
    return launch(kernel, (unsigned)grid, kPace[F32OUT][best].threads, st, p);
  };
  if constexpr (MODE != kGroupedDepth) {
    if (best == kFew) return run(k_matmul_split<1, 1, MODE, F32OUT>);
    if (best == kFew32) return run(k_matmul_split<2, 2, MODE, F32OUT>);
    if (best == kFew48) return run(k_matmul_split<2, 3, MODE, F32OUT>);
  }
  if constexpr (!F32OUT)
    if (best == kMiddle) return run(k_matmul_tile<128, 128, 2, 4, 1, 0, MODE, F32OUT>);
  if (best == kSmall) return run(k_matmul_tile<64, 64, 2, 2, 1, 16, MODE, F32OUT>);
  if (best == kSmallTeams) return run(k_matmul_tile<64, 64, 2, 2, 2, 16, MODE, F32OUT>);
  constexpr int LARGE = F32OUT ? 128 : 256;
  return run(k_matmul_tile<LARGE, LARGE, 2, F32OUT ? 2 : 4, 1, 0, MODE, F32OUT>);
}

template <int MODE>
tfp8_status launch_product(const ProductArgs &p, bool f32, hipStream_t st) {
  return f32 ? launch_product<MODE, true>(p, st) : launch_product<MODE, false>(p, st);
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;  // rows and columns of one operand
constexpr int64_t kMaxLd = (int64_t)1 << 22;          // codes of a row: a tile's offsets fit 31 bits
constexpr int64_t kMaxLds = (int64_t)1 << 20;         // scales of a row

// Checks of one operand [rows, k] (count of them, `next` bytes apart): strides, pointers.
tfp8_status operand_sizes(int64_t rows, int64_t k, int32_t block, int64_t ld, int64_t lds) {
  if (rows < 0 || rows > kMaxRows || k < 0 || k > kMaxLd || k % block != 0) return TFP8_E_SIZE;
  if (ld > kMaxLd || lds > kMaxLds) return TFP8_E_SIZE;
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
  p.a = Operand{a_codes, a_alpha, a_scale, (int32_t)a_ld, (int32_t)a_lds};
  p.b = Operand{b_codes, b_alpha, b_scale, (int32_t)b_ld, (int32_t)b_lds};
  p.m = (int32_t)m;
  p.n = (int32_t)n;
  p.steps = (int32_t)(k / kStep);
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
  p.a = Operand{a_codes, a_alpha, a_scale, (int32_t)a_ld, (int32_t)a_lds};
  p.b = Operand{b_codes, b_alpha, b_scale, (int32_t)b_ld, (int32_t)b_lds};
  p.m = (int32_t)m;
  p.n = (int32_t)n;
  p.steps = (int32_t)(k / kStep);
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
  p.a = Operand{a_codes, a_alpha, a_scale, (int32_t)a_ld, (int32_t)a_lds};
  p.b = Operand{b_codes, b_alpha, b_scale, (int32_t)b_ld, (int32_t)b_lds};
  p.m = (int32_t)m;
  p.n = (int32_t)n;
  p.steps = (int32_t)(k / kStep);
  p.shift = log2_of(block);
  p.offsets = offsets;
  p.groups = groups;
  p.rows = (int32_t)rows;
  p.out = out;
  p.ldc = n;
  return launch_product<kGroupedDepth>(p, f32, (hipStream_t)stream);
}

}  // extern "C"
