// tfp8_moe.hip - a whole layer of gated experts for a few tokens, the experts' weights compressed.
//
//   logits = x R^T,  the top_k largest of each token's,  w = their softmax
//   y[t] = sum over the chosen e of w[t, e] W2_e (silu(W1_e x) * (W3_e x))
//
// What bounds it is the codes of the experts that are hit, each read once: they go from memory to
// registers and into the matrix instructions, with nothing in between but their widening to float16,
// which is exact.  The rotation is orthogonal, so a row of weights in the rotated basis times x
// in the rotated basis is the product, and x and the hidden values are rotated instead of the weights.
// They go into the products as float16, scaled by a power of two for each block so that its largest is
// below 2^15: 11 bits of each value, an eighth of a bfloat16 output's own rounding.  For float32 outputs
// what that rounds off goes in as a second float16: 22 bits.  Sums are float32.  (One power for a whole row
// would cut off blocks far below its largest value, which count where the weights are small beside that.)
//
// Launches, in order:
//   k_moe_scores  router logits in float64 (a choice hangs on them) and the rotated x
//   k_moe_plan    the choice: each token's experts, and their weights
//   k_moe_up      h = silu(W1_e x) * (W3_e x) for each (token, expert) pair
//   k_moe_rotate  h in the rotated basis
//   k_moe_down    y, or where experts are dealt out over workgroups, their shares of it
//   k_moe_join    the sum of the shares
// For one or two tokens k_moe_up chooses and k_moe_down rotates for itself, where that pays: three launches.
//
// Measured, us: one token, 8 of 64 experts of 2048 x 1024 (54 MB) 4 + 12 + 8, 23 a call, where a launch
// that reads 36 MB and first waits for the choice takes 12; 64 tokens, 6 of 64 of 2048 x 1536 (620 MB) scores 6.9, plan
// 4.8, up 79 (5.4 TB/s), rotate 4.8, down 43 (5.3 TB/s), join 4.9, 140 a call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tfp8.h"
#include "tfp8_device.hpp"
#include "tfp8_host.hpp"

namespace tfp8 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kMostTokens = TFP8_MOE_TOKENS;    // a lane each
constexpr int kMostExperts = TFP8_MOE_EXPERTS;  // a thread each of k_moe_plan
static_assert(kMostTokens == 64 && kMostExperts == 512, "one wavefront, one workgroup");

struct MoeArgs {
  const void *x, *router;
  int64_t ldx, ldo;
  bool x_f32, router_f32, wide, rotate, renormalize;  // wide: rows of x and router start at 16 bytes
  int tokens, experts, top_k, k, f, block_shift;      // block = 128 << block_shift
  const uint8_t *up, *down;
  const float *up_alpha, *up_scale, *down_alpha, *down_scale;
  double *logits;         // [tokens][experts]
  int *where;             // [tokens][experts]: the pair's number, t top_k + .., or -1
  int *ids;               // [pairs]: its expert
  float *gates;           // [pairs]
  int *x_exp;             // [tokens][k / block]: blocks are held divided by 2 to this
  int *h_exp;             // [pairs][f / block], as x_exp
  uint16_t *x_hi, *x_lo;  // [tokens][k], rotated, float16
  float *h;               // [pairs][f]
  uint16_t *h_hi, *h_lo;  // [pairs][f], rotated, float16
  float *shares;          // [splits][tokens][k]
  void *out;
  bool out_f32;
  int splits;
};

// By how many powers of two a block is divided whose largest magnitude is m: a rotated value is at most
// sqrt(B) m, and stays below 2^15.  0 for a block of zeros, and for one that is not finite.
template <int B>
__device__ __forceinline__ int block_exponent(float m) {
  if (m == 0.0f || !(m < __builtin_inff())) return 0;
  return exponent_of(m) + (B == 512 ? 5 : 4) - 15;  // sqrt(128) < 2^4, sqrt(256) = 2^4, sqrt(512) < 2^5
}

__device__ __forceinline__ uint16_t bits(_Float16 x) { return __builtin_bit_cast(uint16_t, x); }

// One block of B values, 8 lanes with B / 8 values each, in runs of 8 at 64 g + 8 j: divided by a power of
// two, whose exponent goes to *exp, rotated and split.  Lane j's results are part lane_perm(j) of each run.
template <int B>
__device__ __forceinline__ void rotate_values(float (&v)[B / 8], bool rotate, int *exp, uint16_t *hi,
                                              uint16_t *lo) {
  constexpr int N = B / 8;
  const int j = threadIdx.x & 7;
  int most = 0;  // as integers: a NaN is larger than all
#pragma unroll
  for (int i = 0; i < N; ++i) most = max(most, __float_as_int(fabsf(v[i])));
  const int e = block_exponent<B>(__int_as_float(group_max_i<8>(most)));
  if (j == 0) *exp = e;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = scale2(v[i], -e);
  int at = j;
  if (rotate) {
    fwht_registers<N, 1>(v);
    fwht_lanes<8, N>(v, j);
    const float c = lane_sign<8>(j) * (float)(1.0 / __builtin_sqrt((double)B));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= c;
    at = lane_perm<8>(j);
  }
#pragma unroll
  for (int g = 0; g < N / 8; ++g) {
    u32x4 a, b;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v0 = v[8 * g + 2 * q], v1 = v[8 * g + 2 * q + 1];
      const _Float16 h0 = (_Float16)v0, h1 = (_Float16)v1;
      a[q] = bits(h0) | (uint32_t)bits(h1) << 16;
      const float r0 = v0 - (float)h0, r1 = v1 - (float)h1;  // exact
      b[q] = bits((_Float16)(fabsf(r0) < __builtin_inff() ? r0 : 0.0f)) |
             (uint32_t)bits((_Float16)(fabsf(r1) < __builtin_inff() ? r1 : 0.0f)) << 16;
    }
    *(u32x4 *)(hi + 64 * g + 8 * at) = a;
    if (lo) *(u32x4 *)(lo + 64 * g + 8 * at) = b;
  }
}
template <int B, class LOAD>
__device__ __forceinline__ void load_block(float (&v)[B / 8], LOAD load) {
#pragma unroll
  for (int g = 0; g < B / 64; ++g) load(&v[8 * g], 64 * g + 8 * (threadIdx.x & 7));
}
template <int B, class LOAD>
__device__ __forceinline__ void rotate_block(LOAD load, bool rotate, int *exp, uint16_t *hi, uint16_t *lo) {
  float v[B / 8];
  load_block<B>(v, load);
  rotate_values<B>(v, rotate, exp, hi, lo);
}

// Eight values from p + at on; wide: 16-byte loads.
__device__ __forceinline__ void load8(const void *p, int64_t at, bool f32, bool wide, float *v) {
  if (f32) {
    const float *q = (const float *)p + at;
    if (wide) {
      const f32x4 a = *(const f32x4 *)q, b = *(const f32x4 *)(q + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[i];
    }
  } else {
    const uint16_t *q = (const uint16_t *)p + at;
    if (wide) {
      const u32x4 a = *(const u32x4 *)q;
#pragma unroll
      for (int i = 0; i < 4; ++i) widen_bf16x2(a[i], v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)q[i] << 16);
    }
  }
}

// The first workgroups: a token each, its row rotated.  The others: an expert and up to 8 tokens each,
// four wavefronts dividing k.
constexpr int kScoreTokens = 8;
constexpr int kScoreThreads = 256;

template <int B>
__global__ __launch_bounds__(kScoreThreads) void k_moe_scores(MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int W = kScoreThreads / 64;
  if ((int)blockIdx.x < a.tokens) {
    const int t = blockIdx.x;
    const int64_t row = t * a.ldx;
    for (int b = threadIdx.x >> 3; b < a.k / B; b += kScoreThreads / 8) {
      const int64_t to = (int64_t)t * a.k + (int64_t)b * B;
      rotate_block<B>(
          [&](float *v, int o) { load8(a.x, row + b * B + o, a.x_f32, a.wide, v); }, a.rotate,
          a.x_exp + t * (a.k / B) + b, a.x_hi + to, a.out_f32 ? a.x_lo + to : nullptr);
    }
    return;
  }
  __shared__ double part[W][kScoreTokens];
  const int groups = (a.tokens + kScoreTokens - 1) / kScoreTokens;
  const int at = blockIdx.x - a.tokens, e = at / groups, t0 = at % groups * kScoreTokens;
  double s[kScoreTokens] = {};
  for (int c = 8 * threadIdx.x; c < a.k; c += 8 * kScoreThreads) {
    float r[8];
    load8(a.router, (int64_t)e * a.k + c, a.router_f32, a.wide, r);
#pragma unroll
    for (int i = 0; i < kScoreTokens; ++i) {
      if (t0 + i >= a.tokens) break;
      float x[8];
      load8(a.x, (t0 + i) * a.ldx + c, a.x_f32, a.wide, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[i] = fma((double)r[q], (double)x[q], s[i]);
    }
  }
  // 8 sums over 64 lanes: lanes that exchange keep half of the sums each, until one is left
#pragma unroll
  for (int k = 4, d = 32; k; k >>= 1, d >>= 1)
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const bool high = lane & d;
      const double mine = high ? s[i + k] : s[i], other = high ? s[i] : s[i + k];
      s[i] = mine + __shfl_xor(other, d);
    }
#pragma unroll
  for (int d = 4; d; d >>= 1) s[0] += __shfl_xor(s[0], d);
  if ((lane & 7) == 0) part[w][lane >> 3] = s[0];  // token (bit 5, bit 4, bit 3)
  __syncthreads();
  if (threadIdx.x < kScoreTokens && t0 + (int)threadIdx.x < a.tokens) {
    double l = part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < W; ++i) l += part[i][threadIdx.x];
    a.logits[(int64_t)(t0 + threadIdx.x) * a.experts + e] = l;
  }
}

// A workgroup a token.  An expert's rank is the number of those with a larger logit, or an equal one and a
// lower index, so that exactly top_k are chosen whatever the logits are (NaN counts as infinity).
// EXPERTS threads an expert each, four times over: each of the four compares with a quarter.
template <int EXPERTS>
__global__ __launch_bounds__(EXPERTS >= 256 ? 1024 : 256) void k_moe_plan(MoeArgs a) {
  constexpr int QUARTERS = EXPERTS == 512 ? 2 : 4, W = EXPERTS / 64;
  __shared__ double l[EXPERTS];
  __shared__ int ranks[QUARTERS][EXPERTS];
  __shared__ double top;
  __shared__ float sums[W];
  __shared__ int chosen[W];
  const int t = blockIdx.x, E = a.experts;
  const int e = threadIdx.x % EXPERTS, quarter = threadIdx.x / EXPERTS, lane = e & 63;
  const double logit = e < E ? a.logits[(int64_t)t * E + e] : -__builtin_inf();
  const double mine = logit != logit ? __builtin_inf() : logit;
  if (quarter == 0) l[e] = mine;  // past the last expert: -infinity, at indexes above all
  __syncthreads();
  int rank = 0;
  const int from = quarter * (EXPERTS / QUARTERS);
#pragma unroll 8
  for (int c = from; c < from + EXPERTS / QUARTERS; ++c)
    rank += l[c] > mine || (l[c] == mine && c < e);
  ranks[quarter][e] = rank;
  __syncthreads();
  if (quarter) rank = EXPERTS;
  else {
#pragma unroll
    for (int i = 1; i < QUARTERS; ++i) rank += ranks[i][e];
    if (rank == 0) top = mine;
  }
  const bool in = e < E && rank < a.top_k;
  const uint64_t set = __ballot(in);
  if (quarter == 0 && lane == 0) chosen[e >> 6] = __popcll(set);
  __syncthreads();
  int before = __popcll(set & ((1ull << lane) - 1));
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < e >> 6) before += chosen[i];
  const float power = logit != logit ? __builtin_nanf("") : expf((float)(mine - top));
  float sum = in || (!a.renormalize && quarter == 0 && e < E) ? power : 0.0f;
  sum = group_sum<32>(sum);
  sum += __shfl_xor(sum, 32);
  if (quarter == 0 && lane == 0) sums[e >> 6] = sum;
  __syncthreads();
  if (quarter || e >= E) return;
  sum = sums[0];
#pragma unroll
  for (int i = 1; i < W; ++i) sum += sums[i];
  const int pair = t * a.top_k + before;
  a.where[(int64_t)t * E + e] = in ? pair : -1;
  if (in) {
    a.ids[pair] = e;
    a.gates[pair] = power / sum;
  }
}

// Up to this many tokens k_moe_up chooses and k_moe_down rotates (one token, 8 of 64 experts of 2048 x
// 1024: 23.1 us a call, with launches of their own 25.4; 2 tokens 36.1 and 38.0; 2 tokens, 4 of 16 of
// 1280 x 640: 22.5 and 25.1; for 4 tokens it was 35.5 and 33.9).
constexpr int kAlone = 2;

// The same choice by a workgroup of four wavefronts for itself, for one or two tokens and up to 64 experts.
// Lane e of wavefront w compares expert e of token w % tokens with a quarter or a half of the others.
struct Choice {
  double l[kAlone][64];
  int ranks[4][64], where[kAlone][64], ids[kAlone * 64];
};
static_assert(kAlone == 2, "the wavefronts share the tokens evenly, and a lane's token is its last bit");
__device__ __forceinline__ void choose(const MoeArgs &a, Choice &c, bool tell) {
  const int lane = threadIdx.x & 63, E = a.experts;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = 4 / a.tokens, t = w % a.tokens, part = w / a.tokens;
  const double logit = lane < E ? a.logits[t * E + lane] : -__builtin_inf();
  const double mine = logit != logit ? __builtin_inf() : logit;
  c.l[t][lane] = mine;  // by each part's wavefront, the same
  __syncthreads();
  int rank = 0;
  const int from = part * (64 / parts);
#pragma unroll 8
  for (int o = from; o < from + 64 / parts; ++o)
    rank += c.l[t][o] > mine || (c.l[t][o] == mine && o < lane);
  c.ranks[w][lane] = rank;
  __syncthreads();
  if (part == 0) {
    for (int i = 1; i < parts; ++i) rank += c.ranks[t + i * a.tokens][lane];
    const bool in = lane < E && rank < a.top_k;
    const uint64_t set = __ballot(in), best = __ballot(rank == 0);
    const int pair = t * a.top_k + __popcll(set & ((1ull << lane) - 1));
    c.where[t][lane] = in ? pair : -1;
    if (in) c.ids[pair] = lane;
    if (tell) {  // what k_moe_down needs
      const double top = __shfl(mine, __builtin_ctzll(best));
      const float power = logit != logit ? __builtin_nanf("") : expf((float)(mine - top));
      float sum = in || (!a.renormalize && lane < E) ? power : 0.0f;
      sum = group_sum<32>(sum);
      sum += __shfl_xor(sum, 32);
      if (lane < E) a.where[t * E + lane] = in ? pair : -1;
      if (in) {
        a.ids[pair] = lane;
        a.gates[pair] = power / sum;
      }
    }
  }
  __syncthreads();
}

// --------------------------------------------------------------------------------------------
// Products of a few tokens and 16 rows of weights to a wavefront, by v_mfma_f32_16x16x32_f16: lane l
// = 16 g + n holds token n's values (first operand) and weight row n's (second) at the 8 places 8 g ..
// of 32, and of the sums, tokens 4 g .. 4 g + 3 with row n.  Any order of the places does, the same for
// both: of 128 places lane group g takes 32 g to 32 g + 31, in four instructions.
//
// The vector cache looks up a line for each few neighbouring lanes, so neighbouring lanes load neighbouring
// bytes, and exchange them after: pairs of lanes 32 bytes of a row of codes (a load covers whole lines of
// 8 rows), four lanes 64 bytes of a token's values.  (Each lane loading from its own row, 64 lookups a
// load, was bound by them: 64 tokens, 6 of 64 experts of 2048 x 1536, 223 us against 169.)
//
// Codes and values come in units of 128 places, up to four of them on their way at a time in a ring of
// registers (NM sets of rows: 2 NM KB a unit); the factors of four units are one load a row set, a
// round ahead.

constexpr int kUnit = 128;
template <int NM, bool LO>
constexpr int depth_of() { return LO ? 3 : 4; }  // what the registers hold

template <int NM, bool LO>
struct Unit {
  u32x4 w[NM][2];          // codes: this lane's 16 bytes of rows 2 (n / 2) and 2 (n / 2) + 1
  u32x4 x[LO ? 8 : 4];     // values: its 16 bytes of tokens 4 (n / 4) .. + 3; what they rounded off
};

// Loads go through buffer descriptors: a base that is the same for all lanes (`from` has to be; 2 GB
// from there are in reach), a lane's offset in bytes, and one for all lanes, with no address arithmetic
// in vector registers.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_at(const void *from) {
  const uint64_t p = (uint64_t)from;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), 0, 0x7FFFFFFF, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t lane, int all) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane, all, 0));
}

// Where a lane's parts lie: bases for all lanes, and the lane's offsets in bytes.
//
// H = 2, for up to 8 tokens: a set is 8 rows twice, the second time from unit `span` on of each, and so are the
// tokens.  Of the sums, those of a row's and a token's same half are meant.  Tiles are half as high then, and
// twice as many.
//
// near: the tokens' values lie in LDS.
template <int NM, int H = 1>
struct Rows {
  Buffer codes[NM], alpha[NM], scale[NM], hi, lo, exps;
  const uint16_t *near_hi, *near_lo;
  const int *near_exps;
  uint32_t code, factor, exp;  // of its even row; of row lane / 4; of token lane / 4
  int places;              // from a row to the next
  uint32_t token[4];       // of its four tokens' values
  int span;

  // sets of 16 / H rows from `row` on of an operand with rows of `width` codes in `blocks` blocks
  __device__ __forceinline__ void set(int m, const uint8_t *c, const float *a, const float *s,
                                      int64_t row, int width, int blocks) {
    codes[m] = buffer_at(c + row * width);
    alpha[m] = buffer_at(a + row * blocks);
    scale[m] = buffer_at(s + row * blocks);
    const int lane = threadIdx.x & 63;
    places = width;
    const int even = lane & (H == 2 ? 6 : 14), own = lane >> 2 & (H == 2 ? 7 : 15);
    code = (uint32_t)even * width + 32 * (lane >> 4) + 16 * (lane & 1);
    if (H == 2 && lane & 8) code += span * kUnit;
    factor = (uint32_t)own * blocks * 4;
  }
  // tokens' rows of values: `row` is that of token n here (any row for none: its sums go nowhere)
  template <bool NEAR = false>
  __device__ __forceinline__ void set_tokens(const uint16_t *h, const uint16_t *l, const int *e, int row,
                                             int width, int blocks) {
    const int lane = threadIdx.x & 63;
    if constexpr (NEAR) {
      near_hi = h;
      near_lo = l;
      near_exps = e;
    } else {
      hi = buffer_at(h);
      lo = buffer_at(l);
      exps = buffer_at(e);
    }
    exp = (uint32_t)__shfl(row, lane >> 2) * blocks * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t from = (uint32_t)__shfl(row, (lane & 12) + i) * width;
      if (H == 2 && lane & 8) from += span * kUnit;
      token[i] = (from + 32 * (lane >> 4) + 8 * (lane & 3)) * 2;
    }
  }
};

template <int NM, bool LO, int H, bool NEAR>
__device__ __forceinline__ void load_unit(Unit<NM, LO> &p, const Rows<NM, H> &r, int u) {
  const int at = u * kUnit;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NEAR) {
      p.x[i] = *(const u32x4 *)((const char *)(r.near_hi + at) + r.token[i]);
      if constexpr (LO) p.x[4 + i] = *(const u32x4 *)((const char *)(r.near_lo + at) + r.token[i]);
    } else {
      p.x[i] = load16(r.hi, r.token[i], 2 * at);
      if constexpr (LO) p.x[4 + i] = load16(r.lo, r.token[i], 2 * at);
    }
  }
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p.w[m][i] = load16(r.codes[m], r.code, at + i * r.places);
}

// Lanes of a pair (CTRL: their exchange; odd: this is the second) have a of the first's and b of the
// second's row each: after, this lane has both of its own.
template <int CTRL>
__device__ __forceinline__ void exchange(u32x4 &a, u32x4 &b, bool odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = a[i], y = b[i];  // exchanged by all lanes, then chosen: no branch
    const uint32_t ox = (uint32_t)dpp_i<CTRL>((int)x), oy = (uint32_t)dpp_i<CTRL>((int)y);
    a[i] = odd ? oy : x;
    b[i] = odd ? y : ox;
  }
}

__device__ __forceinline__ f16x8 widen_codes(uint32_t d0, uint32_t d1) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d0, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d0, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d1, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d1, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// total += the unit's products times the rows' factors and 2 to the tokens' exponents, those of row and token n
// in lane 4 n + `from`.
template <int NM, bool LO>
__device__ __forceinline__ void add_unit(f32x4 (&total)[NM], Unit<NM, LO> &p, const float (&f)[NM], int exp,
                                         int from) {
  const int lane = threadIdx.x & 63, n = lane & 15;
  int e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = __shfl(exp, (lane & 48) + 4 * i + from);
#pragma unroll
  for (int k = 0; k < (LO ? 8 : 4); k += 4) {
    exchange<kDppXor1>(p.x[k], p.x[k + 1], lane & 1);
    exchange<kDppXor1>(p.x[k + 2], p.x[k + 3], lane & 1);
    exchange<kDppXor2>(p.x[k], p.x[k + 2], lane & 2);
    exchange<kDppXor2>(p.x[k + 1], p.x[k + 3], lane & 2);
  }
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    exchange<kDppXor1>(p.w[m][0], p.w[m][1], lane & 1);
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x8 w = widen_codes(p.w[m][i / 2][2 * (i & 1)], p.w[m][i / 2][2 * (i & 1) + 1]);
      sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p.x[i]), w, sum, 0, 0, 0);
      if constexpr (LO)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p.x[4 + i]), w, sum, 0,
                                                     0, 0);
    }
    const float fu = __shfl(f[m], 4 * n + from);
#pragma unroll
    for (int i = 0; i < 4; ++i) total[m][i] = fmaf(sum[i], scale2(fu, e[i]), total[m][i]);
  }
}

// The sums over units [u0, u1) of 16 rows of NM sets with up to 16 tokens, in rounds of kDepth units; the
// last round's missing units are the last one again, times 0.  No load hangs on a condition, so that
// the waits are for the oldest unit alone.  H = 2: [u0, u1) is the first half, and `odd` that the second one
// begins with the unit that the first ends with, which counts once.
template <int NM, bool LO, int H, bool NEAR = false>
__device__ __forceinline__ void sum_units(f32x4 (&total)[NM], const Rows<NM, H> &r, int u0, int u1,
                                          int shift, bool odd = false) {
  if (u0 >= u1) return;
  constexpr int kDepth = depth_of<NM, LO>();
  float alpha[NM], scale[NM], f[NM];
  int next_exp, exp;
  const auto load_factors = [&](int u) {  // of units u .. u + 3
    const bool second = H == 2 && threadIdx.x & 32;
    const int mine = u + (int)(threadIdx.x & 3);
    const int b = (min(mine, u1 - 1) + (second ? r.span : 0)) >> shift;
    if constexpr (NEAR)
      next_exp = *(const int *)((const char *)r.near_exps + r.exp + 4 * b);
    else
      next_exp = (int)__builtin_amdgcn_raw_buffer_load_b32(r.exps, r.exp + 4 * b, 0, 0);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      alpha[m] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r.alpha[m], r.factor + 4 * b, 0, 0));
      scale[m] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r.scale[m], r.factor + 4 * b, 0, 0));
      if (mine >= u1 || (second && odd && mine == u0)) scale[m] = 0.0f;
    }
  };
  const auto take_factors = [&] {
#pragma unroll
    for (int m = 0; m < NM; ++m) f[m] = scale[m] * __builtin_amdgcn_rcpf(alpha[m]);
    exp = next_exp;
  };
  Unit<NM, LO> p[kDepth];
  load_factors(u0);
#pragma unroll
  for (int s = 0; s < kDepth; ++s) load_unit<NM, LO, H, NEAR>(p[s], r, min(u0 + s, u1 - 1));
  for (int u = u0 + kDepth; u < u1; u += kDepth) {
    take_factors();
    load_factors(u);
#pragma unroll
    for (int s = 0; s < kDepth; ++s) {
      add_unit<NM, LO>(total, p[s], f, exp, s);
      load_unit<NM, LO, H, NEAR>(p[s], r, min(u + s, u1 - 1));
    }
  }
  take_factors();
#pragma unroll
  for (int s = 0; s < kDepth; ++s) add_unit<NM, LO>(total, p[s], f, exp, s);
}

// Which of a set's tokens is number `nth`, from 0 on; -1 past its last.
__device__ __forceinline__ int nth_token(uint64_t set, int nth) {
  for (int i = 0; i < nth; ++i) set &= set - 1;
  return set ? __builtin_ctzll(set) : -1;
}

// The expert of a slot and where its tokens are.  With fewer pairs than experts a slot is a pair, and
// stands for its expert where its token is the first that chose it; else a slot is an expert.
struct Slot {
  int expert;
  int pair;      // of token `lane`, -1: it has not chosen the expert
  uint64_t set;  // 0: nothing to do
};
__device__ __forceinline__ int slots_of(const MoeArgs &a) { return min(a.tokens * a.top_k, a.experts); }
__device__ __forceinline__ Slot slot_of(const MoeArgs &a, const Choice &c, int slot) {
  const int lane = threadIdx.x & 63;
  const bool by_pair = a.tokens * a.top_k < a.experts;
  Slot s;
  s.expert = by_pair ? __builtin_amdgcn_readfirstlane(c.ids[slot]) : slot;
  s.pair = lane < a.tokens ? c.where[lane & 1][s.expert] : -1;
  s.set = __ballot(s.pair >= 0);
  if (by_pair && s.set && __builtin_ctzll(s.set) != slot / a.top_k) s.set = 0;
  return s;
}
__device__ __forceinline__ Slot slot_of(const MoeArgs &a, int slot) {
  const int lane = threadIdx.x & 63;
  const bool by_pair = a.tokens * a.top_k < a.experts;
  Slot s;
  s.expert = by_pair ? __builtin_amdgcn_readfirstlane(a.ids[slot]) : slot;
  if (by_pair && a.tokens == 1) {  // a slot is a pair of the one token: nothing to look up
    s.pair = lane ? -1 : slot;
    s.set = 1;
    return s;
  }
  s.pair = lane < a.tokens ? a.where[(int64_t)lane * a.experts + s.expert] : -1;
  s.set = __ballot(s.pair >= 0);
  if (by_pair && s.set && __builtin_ctzll(s.set) != slot / a.top_k) s.set = 0;
  return s;
}

// h of one expert's tokens, 16 at a time.  A wavefront takes 16 of the f hidden places, the gate's rows and
// the other's together, so that x is read once for both, and of the four of a workgroup two divide k.  (By
// one and by four, us a call: 2 tokens, 2 of 8 of 4096 x 14336, 158 and 137 against 136; 8 tokens, 6 of 64 of 2048 x
// 1408, 98 and 103 against 95; 64 tokens, 6 of 64 of 2048 x 1536, 142 and 163 against 139.)
constexpr int kUpWaves = 4, kUpParts = 2, kUpTiles = kUpWaves / kUpParts;
template <bool LO, bool CHOOSE>
__global__ __launch_bounds__(64 * kUpWaves, 2) void k_moe_up(MoeArgs a) {
  __shared__ float part[kUpWaves][2][4][64];
  const int tiles = a.f / (16 * kUpTiles);  // f is a multiple of 128
  Slot s;
  if constexpr (CHOOSE) {
    __shared__ Choice choice;
    choose(a, choice, blockIdx.x == 0);
    s = slot_of(a, choice, blockIdx.x / tiles);
  } else {
    s = slot_of(a, blockIdx.x / tiles);
  }
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f0 = (blockIdx.x % tiles * kUpTiles + w / kUpParts) * 16, share = w % kUpParts;
  const int blocks = a.k >> (7 + a.block_shift), units = a.k / kUnit;
  for (int first = 0; first < __popcll(s.set); first += 16) {
    const int token = nth_token(s.set, first + n), safe = token < 0 ? __builtin_ctzll(s.set) : token;
    const int of_token = __shfl(s.pair, safe);  // by all lanes: it reads from those past the set, too
    const int pair = token < 0 ? -1 : of_token;
    f32x4 total[2] = {};
    Rows<2> r;
#pragma unroll
    for (int m = 0; m < 2; ++m)
      r.set(m, a.up, a.up_alpha, a.up_scale, ((int64_t)s.expert * 2 + m) * a.f + f0, a.k, blocks);
    r.set_tokens(a.x_hi, a.x_lo, a.x_exp, safe, a.k, blocks);
    sum_units<2, LO, 1>(total, r, units * share / kUpParts, units * (share + 1) / kUpParts,
                        a.block_shift);
    if (first) __syncthreads();  // the sums of the tokens before are read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[w][m][i][lane] = total[m][i];
    __syncthreads();
    if (share) continue;
#pragma unroll
    for (int k = 1; k < kUpParts; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[m][i] += part[w + k][m][i][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int to = __shfl(pair, 4 * g + i);
      const float gate = total[0][i];
      if (to >= 0) a.h[(int64_t)to * a.f + f0 + n] = gate / (1.0f + expf(-gate)) * total[1][i];
    }
  }
}

// h, 32 blocks a workgroup.
constexpr int kRotateThreads = 256;
template <int B>
__global__ __launch_bounds__(kRotateThreads) void k_moe_rotate(MoeArgs a) {
  const int64_t b = (int64_t)blockIdx.x * (kRotateThreads / 8) + (threadIdx.x >> 3), at = b * B;
  if (at >= (int64_t)a.tokens * a.top_k * a.f) return;
  rotate_block<B>([&](float *v, int o) { load8(a.h, at + o, true, true, v); }, a.rotate, a.h_exp + b,
                  a.h_hi + at, a.out_f32 ? a.h_lo + at : nullptr);
}

// 16 NM / H places of y for all tokens.  Workgroup split s of a.splits takes every a.splits-th slot; its eight
// wavefronts deal out (slot, 16 tokens, part of f), each adding to its own sums in LDS, and the eight
// sums are added in order: no atomics, so that calls agree bit for bit.  With several splits k_moe_join
// adds their shares.  (The last workgroup of a tile to finish added them first, found by a counter
// behind a fence: the fence writes back the whole L2, and one token took 85 us instead of 14.)
__device__ __forceinline__ void store_out(const MoeArgs &a, int t, int at, float y) {
  if (a.out_f32)
    ((float *)a.out)[t * a.ldo + at] = y;
  else
    ((__bf16 *)a.out)[t * a.ldo + at] = (__bf16)y;
}
constexpr int kDownWaves = 8;
//
// B > 0, for up to kNear hidden values in all: every workgroup rotates them for itself, into LDS.
constexpr int kNear = 16384;
template <int NM, int H, int TOKENS, bool LO, int B = 0>
__global__ __launch_bounds__(64 * kDownWaves, 2) void k_moe_down(MoeArgs a) {
  constexpr int R = 16 * NM / H;
  static_assert(H == 1 || TOKENS <= 8, "tokens in halves");
  constexpr bool NEAR = B > 0;
  __shared__ uint16_t near_hi[NEAR ? kNear : 8], near_lo[NEAR && LO ? kNear : 8];
  __shared__ int near_exp[NEAR ? kNear / 128 : 1];
  if constexpr (NEAR) {
    const int all = a.tokens * a.top_k * (a.f / B);
    for (int b = threadIdx.x >> 3; b < all; b += 64 * kDownWaves / 8)
      rotate_block<B>([&](float *v, int o) { load8(a.h, (int64_t)b * B + o, true, true, v); }, a.rotate,
                      near_exp + b, near_hi + b * B, LO ? near_lo + b * B : nullptr);
    __syncthreads();
  }
  __shared__ float sums[kDownWaves][TOKENS][R];
  const int tiles = a.k / R, tile = blockIdx.x % tiles, split = blockIdx.x / tiles;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int t = lane / R; t < a.tokens; t += 64 / R) sums[w][t][lane % R] = 0.0f;
  const int slots = slots_of(a), units = a.f / kUnit, blocks = a.f >> (7 + a.block_shift);
  const int mine = slots > split ? (slots - split + a.splits - 1) / a.splits : 0;
  // few slots: several wavefronts divide one's f
  const int parts = min(mine > 0 && mine < kDownWaves ? kDownWaves / mine : 1, units);
  for (int item = w; item < mine * parts; item += kDownWaves) {
    const int part = item % parts;
    const Slot s = slot_of(a, split + item / parts * a.splits);
    const int u0 = units * part / parts, u1 = units * (part + 1) / parts;
    for (int first = 0; first < __popcll(s.set); first += 16) {
      const int token = nth_token(s.set, first + (H == 2 ? n & 7 : n));
      const int safe = token < 0 ? __builtin_ctzll(s.set) : token;
      const int pair = __shfl(s.pair, safe);
      const float gate = a.gates[pair];
      Rows<NM, H> r;
      const int half = (u1 - u0 + H - 1) / H;  // H = 2: the second half ends where the part does
      r.span = u1 - half - u0;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        r.set(m, a.down, a.down_alpha, a.down_scale, (int64_t)s.expert * a.k + R * tile + 16 * m, a.f,
              blocks);
      if constexpr (NEAR)
        r.template set_tokens<true>(near_hi, near_lo, near_exp, pair, a.f, blocks);
      else
        r.set_tokens(a.h_hi, a.h_lo, a.h_exp, pair, a.f, blocks);
      f32x4 total[NM] = {};
      sum_units<NM, LO, H, NEAR>(total, r, u0, u0 + half, a.block_shift, H == 2 && (u1 - u0) & 1);
      if constexpr (H == 2) {
        // lane (g, n) has token 4 (g % 2) + i's half g / 2 with row n % 8's half n / 8
#pragma unroll
        for (int i = 0; i < 4; ++i) total[0][i] += __shfl_xor(total[0][i], 40);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = __shfl(token, 4 * g + i);
        const float gt = __shfl(gate, 4 * g + i);
        if (t < 0 || (H == 2 && (g > 1 || n > 7))) continue;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          float &to = sums[w][t][16 * m + n];
          to = fmaf(gt, total[m][i], to);
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * R; i += 64 * kDownWaves) {
    const int t = i / R, at = R * tile + i % R;
    float y = sums[0][t][i % R];
#pragma unroll
    for (int k = 1; k < kDownWaves; ++k) y += sums[k][t][i % R];
    if (a.splits > 1)
      a.shares[((int64_t)split * a.tokens + t) * a.k + at] = y;
    else
      store_out(a, t, at, y);
  }
}

__global__ __launch_bounds__(256) void k_moe_join(MoeArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * a.k) return;
  float y = a.shares[i];
  for (int s = 1; s < a.splits; ++s) y += a.shares[(int64_t)s * a.tokens * a.k + i];
  store_out(a, i / a.k, i % a.k, y);
}

}  // namespace tfp8

using namespace tfp8;

namespace {

constexpr int kMostK = 1 << 20;  // of k and f
constexpr int64_t kMostHidden = (int64_t)1 << 29;  // of all pairs: k_moe_up has 8 threads each, below 2^32

// Rows of an output tile of k_moe_down, and how many workgroups share its experts.
// 8 rows where that fills the compute units (one token, 8 of 64 experts of 2048 x 1024: 24.1 us a call
// against 25.1), unless the wavefronts have many slots each, which then take as long to look up as to read
// (8 tokens, 6 of 64 of 2048 x 1408: 94 against 86).  32 rows read a token's values half as often (48
// tokens, 4 of 16 of 2560 x 1024: 64 against 69; 36 tokens, 7 of 10 of 4864 x 3200: 267 against 306; but 64
// tokens, 2 of 8 of 4096 x 2048: 101 against 92).
int down_rows(int64_t tokens, int64_t pairs, int64_t k) {
  if (tokens <= 8 && pairs <= 16 && k < 4096) return 8;
  return pairs >= 192 ? 32 : 16;
}
// Experts are shared out until the compute units are full, as long as each wavefront keeps a slot; and to more
// than half of them where it keeps 8 units of a part of one (52 tokens, 5 of 16 of 384 x 14336, float32: 546 us
// a call without that, 228 with; 18 tokens, 4 of 8 of 768 x 2688: 43 and 38; but to all of them 3 tokens, 4 of 26 of 1536
// x 2048: 44 and 49).
int down_splits(int64_t tokens, int64_t pairs, int64_t experts, int64_t k, int64_t f) {
  const int64_t tiles = k / down_rows(tokens, pairs, k), slots = std::min(pairs, experts);
  const int64_t units = f / kUnit;
  int64_t s = 1;
  while ((s * 2 * kDownWaves <= slots && s * tiles < 256) ||
         (s * 2 <= slots && s * 2 * kDownWaves * 8 < slots * units && s * tiles < 128))
    s *= 2;
  return (int)s;
}

struct MoeSizes {
  int64_t tokens, experts, top_k, k, f;
};
bool sizes_ok(const MoeSizes &s) {
  return s.tokens >= 0 && s.tokens <= kMostTokens && s.experts >= 1 && s.experts <= kMostExperts &&
         s.top_k >= 1 && s.top_k <= s.experts && s.k >= 1 && s.k <= kMostK && s.f >= 1 &&
         s.f <= kMostK && s.tokens * s.top_k * s.f < kMostHidden;
}

// The workspace's parts, each from a multiple of 16 bytes on; base = NULL counts them.
int64_t lay_out(MoeArgs &a, char *base, const MoeSizes &s) {
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    char *p = base + at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  const int64_t pairs = s.tokens * s.top_k;
  a.logits = (double *)take(s.tokens * s.experts * 8);
  a.where = (int *)take(s.tokens * s.experts * 4);
  a.ids = (int *)take(pairs * 4);
  a.gates = (float *)take(pairs * 4);
  a.x_exp = (int *)take(s.tokens * (s.k / kUnit) * 4);
  a.h_exp = (int *)take(pairs * (s.f / kUnit) * 4);
  a.x_hi = (uint16_t *)take(s.tokens * s.k * 2);
  a.x_lo = (uint16_t *)take(s.tokens * s.k * 2);
  a.h = (float *)take(pairs * s.f * 4);
  a.h_hi = (uint16_t *)take(pairs * s.f * 2);
  a.h_lo = (uint16_t *)take(pairs * s.f * 2);
  a.splits = down_splits(s.tokens, pairs, s.experts, s.k, s.f);
  a.shares = (float *)take(a.splits > 1 ? a.splits * s.tokens * s.k * 4 : 0);
  return at;
}

template <bool LO, int B>
tfp8_status launch_down(const MoeArgs &a, int rows, bool near, hipStream_t st) {
  const unsigned grid = (unsigned)(a.k / rows * a.splits);
  constexpr int nt = 64 * kDownWaves;
  if (near)
    return rows == 8 ? launch(k_moe_down<1, 2, 8, LO, B>, grid, nt, st, a)
                     : launch(k_moe_down<1, 1, 16, LO, B>, grid, nt, st, a);
  if (rows == 8) return launch(k_moe_down<1, 2, 8, LO>, grid, nt, st, a);
  if (a.tokens <= 16)
    return rows == 16 ? launch(k_moe_down<1, 1, 16, LO>, grid, nt, st, a)
                      : launch(k_moe_down<2, 1, 16, LO>, grid, nt, st, a);
  return rows == 16 ? launch(k_moe_down<1, 1, kMostTokens, LO>, grid, nt, st, a)
                    : launch(k_moe_down<2, 1, kMostTokens, LO>, grid, nt, st, a);
}

template <int B, bool LO>
tfp8_status launch_layer(const MoeArgs &a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.tokens * a.top_k, slots = std::min<int64_t>(pairs, a.experts);
  const int64_t groups = (a.tokens + kScoreTokens - 1) / kScoreTokens;
  tfp8_status s = launch(k_moe_scores<B>, (unsigned)(a.tokens + a.experts * groups), kScoreThreads, st,
                         a);
  if (s != TFP8_OK) return s;
  const int64_t ups = slots * (a.f / (16 * kUpTiles));  // workgroups of k_moe_up
  // it chooses, unless these are many, each of which would (2 tokens, 2 of 8 experts of 4096 x 14336, 1792
  // workgroups: 102 us against 86)
  const bool choose = a.tokens <= kAlone && a.experts <= 64 && ups <= 512;
  if (!choose) {
    s = a.experts <= 64    ? launch(k_moe_plan<64>, a.tokens, 256, st, a)
        : a.experts <= 256 ? launch(k_moe_plan<256>, a.tokens, 1024, st, a)
                           : launch(k_moe_plan<512>, a.tokens, 1024, st, a);
    if (s != TFP8_OK) return s;
  }
  s = choose ? launch(k_moe_up<LO, true>, (unsigned)ups, 64 * kUpWaves, st, a)
             : launch(k_moe_up<LO, false>, (unsigned)ups, 64 * kUpWaves, st, a);
  if (s != TFP8_OK) return s;
  const int rows = down_rows(a.tokens, pairs, a.k);
  const bool near = a.tokens <= kAlone && a.splits == 1 && pairs * a.f <= kNear;  // k_moe_down rotates
  if (!near) {
    const int64_t blocks = pairs * (a.f / B), per = kRotateThreads / 8;
    s = launch(k_moe_rotate<B>, (unsigned)((blocks + per - 1) / per), kRotateThreads, st, a);
    if (s != TFP8_OK) return s;
  }
  s = launch_down<LO, B>(a, rows, near, st);
  if (s != TFP8_OK || a.splits == 1) return s;
  return launch(k_moe_join, (unsigned)((a.tokens * a.k + 255) / 256), 256, st, a);
}

}  // namespace

extern "C" {

int64_t tfp8_moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t k, int64_t f) {
  const MoeSizes s{tokens, experts, top_k, k, f};
  MoeArgs a{};
  return sizes_ok(s) ? lay_out(a, nullptr, s) : 0;
}

tfp8_status tfp8_moe_layer(const void *x, tfp8_dtype x_dtype, int64_t ldx, const void *router,
                           tfp8_dtype router_dtype, const uint8_t *up_codes, const float *up_alpha,
                           const float *up_scale, const uint8_t *down_codes, const float *down_alpha,
                           const float *down_scale, int64_t tokens, int64_t experts, int64_t top_k,
                           int64_t k, int64_t f, int32_t block, uint32_t flags, void *workspace,
                           int64_t workspace_bytes, void *out, tfp8_dtype out_dtype, int64_t ldo,
                           void *stream) {
  if (block != 128 && block != 256 && block != 512) return TFP8_E_BLOCK;
  const MoeSizes sizes{tokens, experts, top_k, k, f};
  if (!sizes_ok(sizes) || k % block != 0 || f % block != 0) return TFP8_E_SIZE;
  for (const tfp8_dtype d : {x_dtype, router_dtype, out_dtype})
    if (d != TFP8_BF16 && d != TFP8_F32) return TFP8_E_DTYPE;
  if (flags & ~(uint32_t)(TFP8_FLAG_NO_ROTATION | TFP8_MOE_ALL_EXPERTS)) return TFP8_E_ARG;
  if (ldx < k || ldo < k) return TFP8_E_ARG;
  if (ldx > TFP8_MAX_N / kMostTokens || ldo > TFP8_MAX_N / kMostTokens) return TFP8_E_SIZE;
  if (tokens == 0) return TFP8_OK;
  if (!x || !router || !up_codes || !up_alpha || !up_scale || !down_codes || !down_alpha ||
      !down_scale || !workspace || !out)
    return TFP8_E_NULL;
  const int xs = x_dtype == TFP8_F32 ? 4 : 2, rs = router_dtype == TFP8_F32 ? 4 : 2,
            os = out_dtype == TFP8_F32 ? 4 : 2;
  if (!aligned(x, xs) || !aligned(router, rs) || !aligned(up_codes, 16) || !aligned(down_codes, 16) ||
      !aligned(up_alpha, 4) || !aligned(up_scale, 4) || !aligned(down_alpha, 4) ||
      !aligned(down_scale, 4) || !aligned(workspace, 16) || !aligned(out, os))
    return TFP8_E_ALIGN;
  MoeArgs a{};
  const int64_t need = lay_out(a, (char *)workspace, sizes);
  if (workspace_bytes < need) return TFP8_E_SIZE;
  const int64_t up = experts * 2 * f * k, down = experts * k * f;
  const Range ins[] = {range_of(x, ((tokens - 1) * ldx + k) * xs), range_of(router, experts * k * rs),
                       range_of(up_codes, up), range_of(up_alpha, up / block * 4),
                       range_of(up_scale, up / block * 4), range_of(down_codes, down),
                       range_of(down_alpha, down / block * 4), range_of(down_scale, down / block * 4)};
  const Range outs[] = {range_of(workspace, need), range_of(out, ((tokens - 1) * ldo + k) * os)};
  if (overlap(outs[0], outs[1])) return TFP8_E_ARG;
  for (const Range &o : outs)
    for (const Range &i : ins)
      if (overlap(o, i)) return TFP8_E_ARG;
  a.x = x;
  a.router = router;
  a.ldx = ldx;
  a.ldo = ldo;
  a.x_f32 = x_dtype == TFP8_F32;
  a.router_f32 = router_dtype == TFP8_F32;
  a.wide = aligned(x, 16) && aligned(router, 16) && (tokens == 1 || ldx * xs % 16 == 0);
  a.rotate = !(flags & TFP8_FLAG_NO_ROTATION);
  a.renormalize = !(flags & TFP8_MOE_ALL_EXPERTS);
  a.tokens = (int)tokens;
  a.experts = (int)experts;
  a.top_k = (int)top_k;
  a.k = (int)k;
  a.f = (int)f;
  a.block_shift = block == 128 ? 0 : block == 256 ? 1 : 2;
  a.up = up_codes;
  a.up_alpha = up_alpha;
  a.up_scale = up_scale;
  a.down = down_codes;
  a.down_alpha = down_alpha;
  a.down_scale = down_scale;
  a.out = out;
  a.out_f32 = out_dtype == TFP8_F32;
  hipStream_t st = (hipStream_t)stream;
#define TFP8_CASE(BB) return a.out_f32 ? launch_layer<BB, true>(a, st) : launch_layer<BB, false>(a, st)
  switch (block) {
    case 128: TFP8_CASE(128);
    case 256: TFP8_CASE(256);
    default: TFP8_CASE(512);
  }
#undef TFP8_CASE
}

}  // extern "C"
