// tfp8_optimizer.hip - the gradients' norm and the AdamW step, many tensors to a launch.
//
// Both stream: the norm reads each gradient once, the step reads parameter, gradient and states once
// and writes parameter, states and copy once.  Their floor is those bytes.
//
// A launch holds a table of tensors in its kernel arguments (below 4 KB), so that a call copies
// nothing to the device, keeps nothing, and can be captured into a graph.  A workgroup finds its tensor
// by a binary search over the tensors' first workgroups, on scalars.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "../../include/tfp8.h"
#include "tfp8_device.hpp"
#include "tfp8_host.hpp"

namespace tfp8 {

constexpr int kThreads = 256;  // 4 wavefronts a workgroup

template <class T>
__device__ __forceinline__ T ld_stream(const T *p) {
  return __builtin_nontemporal_load(p);
}
template <class T>
__device__ __forceinline__ void st_stream(T v, T *p) {
  __builtin_nontemporal_store(v, p);
}

// Index of the last of `count` ascending first[] that is at most x (0 if none is).
template <class E>
__device__ __forceinline__ int entry_of(const E *e, int count, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int s = 64; s; s >>= 1)
    if (lo + s < count && e[lo + s].first <= x) lo += s;
  return lo;
}

// --------------------------------------------------------------------------------------------
// The norm.  A workgroup takes units of 16 KB (kLoads 16-byte loads a lane, all under way at once),
// every gridDim.x-th of the launch's, and writes one float64 partial sum; k_norm_finish adds the
// partial sums in order.  No atomics: the order hangs on the sizes alone, so that repeated calls agree
// bit for bit.  Bound by memory: 451 MB of bfloat16 in 69 us (6.5 TB/s; part of it lies in the 256 MB
// cache), 285 MB of codes in 46 us (6.2).  Units of 8192 elements, 1024 or 2048 workgroups and 4 or 6
// wavefronts a SIMD are within 3% of each other.  The finish takes 4 us, most of it a launch's own time (its
// four loads one after the other: 0.4 more).

constexpr int kLoads = 4;
constexpr int kUnitBytes = 16 * kLoads * kThreads;
__host__ __device__ inline int unit_elements(int64_t dtype) {
  return dtype == TFP8_F32 ? kUnitBytes / 4 : dtype == TFP8_BF16 ? kUnitBytes / 2 : kUnitBytes;
}
constexpr int kNormGrid = 1024;      // 4 workgroups on each of 256 compute units: all resident
constexpr int kNormTensors = 80;

struct NormEntry {
  const void *data;
  const float *alpha, *scale;
  int64_t n, first;  // first: units of the tensors before it
  int64_t dtype;
};
struct NormTable {
  NormEntry e[kNormTensors];
  int count, block_shift;
  int64_t units;
};

// Sums of squares of a lane's few values: float32, and float64 where that leaves float32's range.
__device__ __forceinline__ bool sum_in_range(float ss) {
  return ss >= 0x1p-80f && ss < __builtin_inff();
}

template <bool F32>
__device__ __forceinline__ double squares(const u32x4 (&d)[kLoads]) {
  float ss = 0.0f;
  double s = 0.0;
  const auto each = [&](auto add) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          add(__uint_as_float(d[k][i]));
        } else {
          float lo, hi;
          widen_bf16x2(d[k][i], lo, hi);
          add(lo);
          add(hi);
        }
      }
  };
  each([&](float x) { ss = fmaf(x, x, ss); });
  if (sum_in_range(ss)) return (double)ss;
  each([&](float x) { s = fma((double)x, (double)x, s); });
  return s;
}

// 16 codes of one block: (s / alpha)^2 sum dec^2.  The rotation is orthogonal, so the block's values
// have the same sum of squares.
__device__ __forceinline__ double squares_codes(u32x4 d, float a, float s) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    unpack_fp8x4(d[i], v[0], v[1], v[2], v[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) ss = fmaf(v[k], v[k], ss);
  }
  const double r = (double)(s * __builtin_amdgcn_rcpf(a));
  return r * r * (double)ss;
}

// Unit u of a tensor, this lane's part: 16-byte loads side by side over the workgroup.  A last unit
// that is not whole goes load by load, its last values one by one.
__device__ __forceinline__ double unit_squares(const NormEntry &e, int64_t u, int shift) {
  const int64_t base = u * unit_elements(e.dtype), left = e.n - base;
  const int t = threadIdx.x;
  u32x4 d[kLoads];
  if (e.dtype == TFP8_CODES) {
    const uint8_t *x = (const uint8_t *)e.data + base;
    const int64_t b0 = base >> shift;
    float a[kLoads], sc[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int at = 16 * (t + kThreads * k);
      const bool in = at < left;  // whole blocks: 16 codes are in or out together
      d[k] = in ? ld_stream((const u32x4 *)(x + at)) : u32x4{0, 0, 0, 0};
      a[k] = in ? e.alpha[b0 + (at >> shift)] : 1.0f;
      sc[k] = in ? e.scale[b0 + (at >> shift)] : 0.0f;
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) s += squares_codes(d[k], a[k], sc[k]);
    return s;
  }
  const bool f32 = e.dtype == TFP8_F32;
  const int per = f32 ? 4 : 8, es = 16 / per;  // elements a load, bytes an element
  const char *x = (const char *)e.data + base * es;
  if (left >= per * kThreads * kLoads) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) d[k] = ld_stream((const u32x4 *)(x + 16 * (t + kThreads * k)));
  } else {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      d[k] = u32x4{0, 0, 0, 0};
      const int at = per * (t + kThreads * k);
      if (at + per <= left) {
        d[k] = ld_stream((const u32x4 *)(x + (int64_t)at * es));
      } else if (f32) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (at + i < left) d[k][i] = ((const uint32_t *)x)[at + i];
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (at + i < left) d[k][i / 2] |= (uint32_t)((const uint16_t *)x)[at + i] << 16 * (i & 1);
      }
    }
  }
  return f32 ? squares<true>(d) : squares<false>(d);
}

// Sum over the workgroup, in a fixed order; thread 0 has it.
__device__ __forceinline__ double workgroup_sum(double s) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

__global__ __launch_bounds__(kThreads) void k_norm(NormTable t, double *partial) {
  double s = 0.0;
  for (int64_t u = blockIdx.x; u < t.units; u += gridDim.x) {
    const NormEntry &e = t.e[entry_of(t.e, t.count, u)];
    s += unit_squares(e, u - e.first, t.block_shift);
  }
  s = workgroup_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void k_norm_finish(const double *partial, int64_t count,
                                                          float max_norm, float *norm, float *scale) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += 4 * kThreads) {
    double d[4];  // four loads under way at once
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = partial[i + k * kThreads < count ? i + k * kThreads : i];
#pragma unroll
    for (int k = 0; k < 4; ++k) s += i + k * kThreads < count ? d[k] : 0.0;
  }
  s = workgroup_sum(s);
  if (threadIdx.x == 0) {
    const double n = sqrt(s), c = (double)max_norm / (n + 1e-6);
    *norm = (float)n;
    // a norm that is infinite, as the float32 that the caller sees, or NaN clips nothing: the step is
    // to be left out
    *scale = (float)n < __builtin_inff() ? (float)(c < 1.0 ? c : 1.0) : __builtin_nanf("");
  }
}

// --------------------------------------------------------------------------------------------
// The step.

// 32 bits of x, each of which depends on all of it: shifts spread the high bits down, odd multipliers
// (2^32 over the golden ratio, and the fraction of the square root of 2) the low ones up.
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ x >> 16;
}
__host__ __device__ inline uint32_t step_key(uint64_t seed, int64_t step) {
  uint32_t k = mix32((uint32_t)seed);
  k = mix32(k ^ (uint32_t)(seed >> 32));
  k = mix32(k ^ (uint32_t)step);
  return mix32(k ^ (uint32_t)((uint64_t)step >> 32));
}

// What a step multiplies by.
struct Factors {
  float keep, rate, root;  // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  uint32_t key;            // of the random bits
};
__host__ __device__ inline double power(double b, int64_t t) {
  double r = 1.0;
  for (; t; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}
__host__ __device__ inline Factors factors_of(double lr, double beta1, double beta2, double decay,
                                              int64_t step, uint64_t seed) {
  Factors f;
  f.keep = (float)(1.0 - lr * decay);
  f.rate = (float)(lr / (1.0 - power(beta1, step)));
  f.root = (float)(1.0 / sqrt(1.0 - power(beta2, step)));
  f.key = step_key(seed, step);
  return f;
}

// The factors where lr or the step lie on the device (a captured step): computed once, not by every
// wavefront.
__global__ void k_adamw_factors(double lr, double beta1, double beta2, double decay, int64_t step,
                                uint64_t seed, const float *lr_dev, const int64_t *step_dev,
                                Factors *out) {
  if (threadIdx.x || blockIdx.x) return;
  if (lr_dev) lr = (double)*lr_dev;
  if (step_dev) step = *step_dev < 1 ? 1 : *step_dev;
  *out = factors_of(lr, beta1, beta2, decay, step, seed);
}

template <bool CODES>
struct StepEntry;
template <>
struct StepEntry<false> {
  void *param;
  const void *grad;
  void *copy;
  int64_t n, start, first;  // first: workgroups of the tensors before it
};
template <>
struct StepEntry<true> {
  void *param;
  const void *grad;
  void *copy;
  int64_t n, start, first;
  const float *grad_alpha, *grad_scale;
  float *copy_alpha, *copy_scale;
};
constexpr int kTableBytes = 3840;
template <bool CODES>
struct StepTable {
  static constexpr int kMost = kTableBytes / sizeof(StepEntry<CODES>);
  StepEntry<CODES> e[kMost];
};
static_assert(StepTable<false>::kMost == 80 && StepTable<true>::kMost == 48, "entries");
static_assert(kNormTensors <= 128 && StepTable<false>::kMost <= 128, "entry_of's search");

struct StepArgs {
  const void *m, *v;
  const float *m_scale, *v_scale;
  void *m_out, *v_out;  // may be the inputs: a tile's states are read before any is written
  float *m_scale_out, *v_scale_out;
  const Factors *factors;  // NULL: f
  const float *grad_scale;
  Factors f;
  float beta1, rest1, eps;          // rest = 1 - beta
  float beta2, root2, root_rest2;   // root: square root of
  int count;
};

// E4M3 codes of four values, |x| <= 448, rounded by v_cvt_sr_fp8_f32: it adds 20 random bits below the
// code's last and cuts (compared with that arithmetic on 2^27 values: the same, save that a subnormal
// code's value is cut to those 20 bits first).  16 random bits and a half are enough: a step of 2^-16 of
// a code.  16 bits of a hash serve the first moment and 16 the second.
template <int PLACE>
__device__ __forceinline__ uint32_t code_into(uint32_t codes, float x, uint32_t random32) {
  return __builtin_amdgcn_cvt_sr_fp8_f32(x, random32, codes, PLACE);
}
template <class F>
__device__ __forceinline__ uint32_t codes_of(const float *x, F random32) {
  uint32_t c = code_into<0>(0, x[0], random32(0));
  c = code_into<1>(c, x[1], random32(1));
  c = code_into<2>(c, x[2], random32(2));
  return code_into<3>(c, x[3], random32(3));
}
constexpr float kSmallestCode = 0x1p-9f;

__device__ __forceinline__ uint32_t bf16_rounded(float x, uint32_t random16) {
  const uint32_t u = __float_as_uint(x);
  return (fabsf(x) < __builtin_inff() ? u + random16 : u) >> 16;
}
__device__ __forceinline__ uint32_t bf16_nearest(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// The square root by hardware, which takes a subnormal value for 0: such a one is scaled first, by a power of 4.
__device__ __forceinline__ float root_of(float v) {
  const bool small = v < 0x1p-126f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.0f);
}

// Four neighbouring elements, as they lie in memory, where `rem` of them are there.
template <bool WHOLE>
__device__ __forceinline__ u32x4 load4_f32(const float *p, int rem) {
  if (WHOLE || rem >= 4) return ld_stream((const u32x4 *)p);
  u32x4 d = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) d[i] = ((const uint32_t *)p)[i];
  return d;
}
template <bool WHOLE>
__device__ __forceinline__ u32x2 load4_bf16(const uint16_t *p, int rem) {
  if (WHOLE || rem >= 4) return ld_stream((const u32x2 *)p);
  u32x2 d = {0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) d[i / 2] |= (uint32_t)p[i] << 16 * (i & 1);
  return d;
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t load4_codes(const uint8_t *p, int rem) {
  if (WHOLE || rem >= 4) return ld_stream((const uint32_t *)p);
  uint32_t d = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) d |= (uint32_t)p[i] << 8 * i;
  return d;
}
__device__ __forceinline__ void store4(float *p, u32x4 d, int rem) {
  if (rem >= 4) return st_stream(d, (u32x4 *)p);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) ((uint32_t *)p)[i] = d[i];
}
__device__ __forceinline__ void store4(uint16_t *p, u32x2 d, int rem) {
  if (rem >= 4) return st_stream(d, (u32x2 *)p);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) p[i] = (uint16_t)(d[i / 2] >> 16 * (i & 1));
}
__device__ __forceinline__ void store4(uint8_t *p, uint32_t d, int rem) {
  if (rem >= 4) return st_stream(d, (uint32_t *)p);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < rem) p[i] = (uint8_t)(d >> 8 * i);
}

// The largest of the magnitudes that G neighbouring lanes hold, for 64 lanes too.
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (G <= 32) {
    return group_max<G>(v);
  } else {
    const int h = group_max_i<32>(__float_as_int(v));
    const int a = __builtin_amdgcn_readlane(h, 0), b = __builtin_amdgcn_readlane(h, 32);
    return __int_as_float(a > b ? a : b);
  }
}

// Where a wavefront's 64 lanes hold the quads (four neighbouring elements) of its tile.
//  Streams: quad q of lane l is elements 256 q + 4 l of a tile of 1024, every access one contiguous
//   piece; a block of B lies over B / 4 lanes (two quads of all 64 at B = 512).
//  Rotated (a gradient or a copy in codes): a block lies in L lanes, quads in the order of compress's
//   float32 line layout, so that its transforms apply.  In lane j the transform leaves the result's
//   part lane_perm(j) of what lane j held as part j.  Of what it held as part lane_perm(j) = P j (linear
//   on the bits of j) it leaves part P^T P j: with p = j0 ^ j1 ^ j2, bits p, j1 ^ p and j0 ^ p.
// Codes in that order are 4 bytes a lane and quad, 32 neighbouring bytes of a line: states read and
// written so ran at 4.3 TB/s, others at 5.8.  So they are exchanged: of the 16 L codes of four quads,
// lane j loads and stores 16 neighbouring ones, from 16 chunk_of(j) on.  Four lanes and four quads are
// transposed.  Where parts are in lane_perm's order (ORDER = 1), two of the four codes then lie 4 lanes
// away, and in P^T P's (2) the upper four lanes hold theirs backwards as well.
template <int L>
__device__ __forceinline__ int chunk_of(int j) {
  return L == 8 ? 2 * (j & 3) + (j >> 2) : j;
}
__device__ __forceinline__ uint32_t from_lane4(uint32_t v) {  // lane j reads lane j ^ 4 = (j ^ 7) ^ 3
  constexpr int kDppXor3 = 0x1B;  // quad_perm [3,2,1,0]
  return (uint32_t)dpp_i<kDppHalfMirror>(dpp_i<kDppXor3>((int)v));
}
__device__ __forceinline__ void transpose4(uint32_t *c, int j) {
  const auto pair = [&](auto ctrl, uint32_t &a, uint32_t &b, bool odd) {
    const uint32_t x = a, y = b;
    const uint32_t ox = (uint32_t)dpp_i<decltype(ctrl)::value>((int)x);
    const uint32_t oy = (uint32_t)dpp_i<decltype(ctrl)::value>((int)y);
    a = odd ? oy : x;
    b = odd ? y : ox;
  };
  constexpr std::integral_constant<int, kDppXor1> by1{};
  constexpr std::integral_constant<int, kDppXor2> by2{};
  pair(by1, c[0], c[1], j & 1);
  pair(by1, c[2], c[3], j & 1);
  pair(by2, c[0], c[2], j & 2);
  pair(by2, c[1], c[3], j & 2);
}
template <int ORDER>
__device__ __forceinline__ void chunks_to_quads(uint32_t *c, int j) {
  static_assert(ORDER < 2, "written only");
  if constexpr (ORDER == 1) {
    c[1] = from_lane4(c[1]);
    c[2] = from_lane4(c[2]);
  }
  transpose4(c, j);
}
template <int ORDER>
__device__ __forceinline__ u32x4 quads_to_chunks(uint32_t *c, int j) {
  transpose4(c, j);
  if constexpr (ORDER > 0) {
    c[1] = from_lane4(c[1]);
    c[2] = from_lane4(c[2]);
  }
  if (ORDER == 2 && j & 4) return u32x4{c[3], c[2], c[1], c[0]};
  return u32x4{c[0], c[1], c[2], c[3]};
}

// A wavefront's copy of n bytes from byte `at` on, a multiple of 4, unless they are there already.
__device__ __forceinline__ void keep_bytes(const void *from, void *to, int64_t at, int n, int lane) {
  if (from == to) return;
  for (int i = 4 * lane; i < n; i += 256) {
    if (i + 4 <= n)
      *(uint32_t *)((char *)to + at + i) = *(const uint32_t *)((const char *)from + at + i);
    else
      for (int k = i; k < n; ++k) ((char *)to)[at + k] = ((const char *)from)[at + k];
  }
}

constexpr int kGradBf16 = TFP8_BF16, kGradF32 = TFP8_F32, kGradCodes = TFP8_CODES;

template <int B, bool PF32, int GT, int BITS, bool CC>
__global__ __launch_bounds__(kThreads) void k_adamw(StepTable<(GT == kGradCodes || CC)> t,
                                                    StepArgs a) {
  constexpr bool ROT = GT == kGradCodes || CC;
  constexpr int L = lanes_per_block(B);
  constexpr int NQ = ROT ? B / (4 * L) : 4;        // quads a lane
  constexpr int N = 4 * NQ;
  constexpr int TE = 64 * N;                       // elements of a wavefront's tile
  constexpr int QB = ROT ? NQ : (B == 512 ? 2 : 1);  // quads of a lane in one block
  constexpr int NB = NQ / QB;                      // blocks that a lane has a part of
  constexpr int G = ROT ? L : (B >= 256 ? 64 : B / 4);  // lanes that share a block
  constexpr int ORDER = GT == kGradCodes && L == 8;  // of parameters and states
  constexpr bool RANDOM = BITS == 8 || !PF32;

  const auto &e = t.e[entry_of(t.e, a.count, blockIdx.x)];
  const int lane = threadIdx.x & 63;
  const int64_t tile = (blockIdx.x - e.first) * (kThreads / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t base = tile * TE;
  if (base >= e.n) return;
  const int left = e.n - base < TE ? (int)(e.n - base) : TE;
  const bool whole = left == TE;
  float c = 1.0f;
  if (a.grad_scale) {
    c = *a.grad_scale;
    if (!(fabsf(c) < __builtin_inff())) {  // the step is left out: new states are the old ones
      const int64_t s0 = e.start + base;
      keep_bytes(a.m, a.m_out, s0 * (BITS / 8), left * (BITS / 8), lane);
      keep_bytes(a.v, a.v_out, s0 * (BITS / 8), left * (BITS / 8), lane);
      if constexpr (BITS == 8) {
        keep_bytes(a.m_scale, a.m_scale_out, s0 / B * 4, (left + B - 1) / B * 4, lane);
        keep_bytes(a.v_scale, a.v_scale_out, s0 / B * 4, (left + B - 1) / B * 4, lane);
      }
      return;
    }
  }
  const Factors f = a.factors ? *a.factors : a.f;

  const int j = lane & (L - 1), bw = lane / L;
  const int at_p = GT == kGradCodes ? lane_perm<L>(j) : j;
  // blocks past the tensor's end (rotated) read the last block and store nothing
  const int bw_in = ROT && bw * B >= left ? (left - 1) / B : bw;
  const auto off = [&](int q, int part, int block) {
    return ROT ? block * B + 8 * L * (q >> 1) + 4 * L * (q & 1) + 4 * part : 256 * q + 4 * lane;
  };
  const auto rem = [&](int o) { return ROT ? (bw * B < left ? 4 : 0) : left - o; };
  const int64_t state0 = e.start + base;  // this tile's first state
  // block k of this lane, from the tile's first
  const auto block_of = [&](int k) {
    const int b = ROT ? bw_in : (256 * QB * k + 4 * lane) / B;
    const int last = (left - 1) / B;
    return b < last ? b : last;
  };

  u32x4 pd[NQ], gd[GT == kGradCodes ? 1 : NQ], gc[GT == kGradCodes ? NQ / 4 : 1];
  u32x4 md[BITS == 32 ? NQ : 1], vd[BITS == 32 ? NQ : 1];
  uint32_t mc[BITS == 8 ? NQ : 1], vc[BITS == 8 ? NQ : 1];
  float ms[NB], vs[NB];
  float ga = 1.0f, gs = 0.0f;
  const auto load = [&](auto is_whole) {
    constexpr bool W = decltype(is_whole)::value;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int op = off(q, at_p, bw_in);
      const int r = W || ROT ? 4 : left - op;
      if constexpr (GT == kGradF32) {
        gd[q] = load4_f32<W || ROT>((const float *)e.grad + base + op, r);
      } else if constexpr (GT == kGradBf16) {
        const u32x2 d = load4_bf16<W || ROT>((const uint16_t *)e.grad + base + op, r);
        gd[q][0] = d[0];
        gd[q][1] = d[1];
      } else if (q % 4 == 0) {
        gc[q / 4] = ld_stream((const u32x4 *)((const uint8_t *)e.grad + base + bw_in * B +
                                              16 * L * (q / 4) + 16 * chunk_of<L>(j)));
      }
      if constexpr (PF32) {
        pd[q] = load4_f32<W || ROT>((const float *)e.param + base + op, r);
      } else {
        const u32x2 d = load4_bf16<W || ROT>((const uint16_t *)e.param + base + op, r);
        pd[q][0] = d[0];
        pd[q][1] = d[1];
      }
      if constexpr (BITS == 8 && ROT) {
        if (q % 4 == 0) {
          const int at = bw_in * B + 16 * L * (q / 4) + 16 * chunk_of<L>(j);
          const u32x4 m4 = ld_stream((const u32x4 *)((const uint8_t *)a.m + state0 + at));
          const u32x4 v4 = ld_stream((const u32x4 *)((const uint8_t *)a.v + state0 + at));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mc[q + i] = m4[i];
            vc[q + i] = v4[i];
          }
        }
      } else if constexpr (BITS == 8) {
        mc[q] = load4_codes<W || ROT>((const uint8_t *)a.m + state0 + op, r);
        vc[q] = load4_codes<W || ROT>((const uint8_t *)a.v + state0 + op, r);
      } else {
        md[q] = load4_f32<W || ROT>((const float *)a.m + state0 + op, r);
        vd[q] = load4_f32<W || ROT>((const float *)a.v + state0 + op, r);
      }
    }
  };
  if (whole || ROT)
    load(std::true_type{});
  else
    load(std::false_type{});
  if constexpr (BITS == 8) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      ms[k] = a.m_scale[state0 / B + block_of(k)];
      vs[k] = a.v_scale[state0 / B + block_of(k)];
    }
  }
  if constexpr (GT == kGradCodes) {
    ga = e.grad_alpha[base / B + bw_in];
    gs = e.grad_scale[base / B + bw_in];
  }

  // the gradient, but for a factor that its block shares, which goes into beta's complements
  float g[N], factor = c;
  if constexpr (GT == kGradCodes) {
#pragma unroll
    for (int k = 0; k < NQ / 4; ++k) {
      uint32_t c[4] = {gc[k][0], gc[k][1], gc[k][2], gc[k][3]};
      chunks_to_quads<0>(c, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float *v = &g[16 * k + 4 * i];
        unpack_fp8x4(c[i], v[0], v[1], v[2], v[3]);
      }
    }
    fwht_registers<N, 1>(g);
    fwht_lanes<L, N>(g, j);
    factor = c * (lane_sign<L>(j) * (gs * (float)(1.0 / __builtin_sqrt((double)B))) *
                  __builtin_amdgcn_rcpf(ga));
  } else {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if constexpr (GT == kGradF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[4 * q + i] = __uint_as_float(gd[q][i]);
      } else {
        widen_bf16x2(gd[q][0], g[4 * q], g[4 * q + 1]);
        widen_bf16x2(gd[q][1], g[4 * q + 2], g[4 * q + 3]);
      }
    }
  }
  const float to_m = factor * a.rest1, to_v = factor * a.root_rest2;
  float old_m[NB], old_v[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    old_m[k] = BITS == 8 ? a.beta1 * ms[k] : a.beta1;
    old_v[k] = BITS == 8 ? a.root2 * vs[k] : a.beta2;
  }

  // the random bits' key: the upper half of a state's index is the tile's or one more
  const uint32_t lo0 = (uint32_t)state0;
  uint32_t key0 = 0, key1 = 0;
  if constexpr (RANDOM) {
    key0 = mix32(f.key ^ (uint32_t)((uint64_t)state0 >> 32));
    key1 = mix32(f.key ^ ((uint32_t)((uint64_t)state0 >> 32) + 1));
  }
  const auto random = [&](int o, int i) {
    const uint32_t lo = lo0 + (uint32_t)o;
    return mix32(lo + i + (lo < lo0 ? key1 : key0));
  };

  float m1[N], r1[N], p1[CC ? N : 1];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int o = off(q, at_p, bw), oi = off(q, at_p, bw_in), left4 = rem(o);
    float p[4], m[4], v[4], x[4];
    if constexpr (PF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = __uint_as_float(pd[q][i]);
    } else {
      widen_bf16x2(pd[q][0], p[0], p[1]);
      widen_bf16x2(pd[q][1], p[2], p[3]);
    }
    if constexpr (BITS == 8) {
      if constexpr (ROT)
        if (q % 4 == 0) {
          chunks_to_quads<ORDER>(&mc[q], j);
          chunks_to_quads<ORDER>(&vc[q], j);
        }
      unpack_fp8x4(mc[q], m[0], m[1], m[2], m[3]);
      unpack_fp8x4(vc[q], v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = __uint_as_float(md[q][i]);
        v[i] = __uint_as_float(vd[q][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // m' = beta1 m + (1 - beta1) g, v' = (sqrt(beta2) r)^2 + (sqrt(1 - beta2) g)^2 (32 bits: beta2 v)
      const float gv = g[4 * q + i] * to_v;
      m[i] = fmaf(g[4 * q + i], to_m, m[i] * old_m[q / QB]);
      v[i] *= old_v[q / QB];
      float r;
      if constexpr (BITS == 8) {  // scaled: the squares may leave float32's range where the root does not
        const int k = exponent_of(fmaxf(fabsf(v[i]), fabsf(gv)));
        const float old = scale2(v[i], -k), now = scale2(gv, -k);
        r = scale2(__builtin_amdgcn_sqrtf(fmaf(now, now, old * old)), k);
      } else {
        v[i] = fmaf(gv, gv, v[i]);
        r = root_of(v[i]);
      }
      const float u = m[i] * __builtin_amdgcn_rcpf(fmaf(r, f.root, a.eps));
      x[i] = fmaf(-f.rate, u, p[i] * f.keep);
      m1[4 * q + i] = m[i];
      r1[4 * q + i] = r;
      if constexpr (CC) p1[4 * q + i] = x[i];
    }
    if constexpr (PF32) {
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(x[i]);
      store4((float *)e.param + base + o, d, left4);
    } else {
      u32x2 d;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = bf16_rounded(x[2 * i], random(oi, 2 * i) >> 8 & 0xFFFFu) |
               bf16_rounded(x[2 * i + 1], random(oi, 2 * i + 1) >> 8 & 0xFFFFu) << 16;
      store4((uint16_t *)e.param + base + o, d, left4);
    }
    if constexpr (!CC) {
      if (e.copy) {
        u32x2 d;
#pragma unroll
        for (int i = 0; i < 2; ++i) d[i] = bf16_nearest(x[2 * i]) | bf16_nearest(x[2 * i + 1]) << 16;
        store4((uint16_t *)e.copy + base + o, d, left4);
      }
    }
    if constexpr (BITS == 32) {
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(m[i]);
      store4((float *)a.m_out + state0 + o, d, left4);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(v[i]);
      store4((float *)a.v_out + state0 + o, d, left4);
    }
  }

  if constexpr (BITS == 8) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      float mm = 0.0f, rm = 0.0f;
#pragma unroll
      for (int i = 4 * QB * k; i < 4 * QB * (k + 1); ++i) {  // a NaN stays one, here and over the lanes
        mm = __builtin_elementwise_maximum(mm, fabsf(m1[i]));
        rm = __builtin_elementwise_maximum(rm, fabsf(r1[i]));
      }
      mm = lanes_max<G>(fabsf(mm));
      rm = lanes_max<G>(fabsf(rm));
      const float im = mm < 0x1p-100f ? 0.0f : 448.0f * __builtin_amdgcn_rcpf(mm);
      const float ir = rm < 0x1p-100f ? 0.0f : 448.0f * __builtin_amdgcn_rcpf(rm);
#pragma unroll
      for (int q = QB * k; q < QB * (k + 1); ++q) {
        const int o = off(q, at_p, bw), oi = off(q, at_p, bw_in), left4 = rem(o);
        uint32_t h[4];
        float m[4], r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = random(oi, i);
          m[i] = __builtin_amdgcn_fmed3f(m1[4 * q + i] * im, -448.0f, 448.0f);
          r[i] = r1[4 * q + i] > 0.0f && !(rm < 0x1p-100f)
                     ? __builtin_amdgcn_fmed3f(r1[4 * q + i] * ir, kSmallestCode, 448.0f) : 0.0f;
        }
        const uint32_t dm = codes_of(m, [&](int i) { return h[i] << 16 | 0x8000u; });
        const uint32_t dv = codes_of(r, [&](int i) { return (h[i] & 0xFFFF0000u) | 0x8000u; });
        if constexpr (ROT) {
          mc[q] = dm;
          vc[q] = dv;
          if (q % 4 == 3) {
            const u32x4 m4 = quads_to_chunks<ORDER>(&mc[q - 3], j);
            const u32x4 v4 = quads_to_chunks<ORDER>(&vc[q - 3], j);
            const int at = bw * B + 16 * L * (q / 4) + 16 * chunk_of<L>(j);
            if (left4 > 0) {
              st_stream(m4, (u32x4 *)((uint8_t *)a.m_out + state0 + at));
              st_stream(v4, (u32x4 *)((uint8_t *)a.v_out + state0 + at));
            }
          }
        } else {
          store4((uint8_t *)a.m_out + state0 + o, dm, left4);
          store4((uint8_t *)a.v_out + state0 + o, dv, left4);
        }
      }
      const bool first = ROT ? j == 0 && bw * B < left
                             : lane % G == 0 && 256 * QB * k + 4 * lane < left;
      if (first) {
        a.m_scale_out[state0 / B + block_of(k)] = mm < 0x1p-100f ? 0.0f : mm * (1.0f / 448.0f);
        a.v_scale_out[state0 / B + block_of(k)] = rm < 0x1p-100f ? 0.0f : rm * (1.0f / 448.0f);
      }
    }
  }

  if constexpr (CC) {  // the new parameters compressed, as compress does (target 1)
    constexpr double kB = (double)B;
    const float ss = group_sum<L>(sum_squares<N>(p1));
    fwht_registers<N, 1>(p1);
    fwht_lanes<L, N>(p1, j);
    float mm = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) mm = fmaxf(mm, fabsf(p1[i]));
    const float M = group_max<L>(mm);
    const float invC = (float)(1.0 / (448.0 * __builtin_sqrt(kB)));
    float cm = 0.0f, alpha = 1.0f, s = 0.0f;
    if (M >= 0x1p-40f && M <= 0x1p60f) {
      alpha = fminf(fmaxf((float)__builtin_sqrt(kB) * __builtin_amdgcn_rsqf(ss), 0x1p-126f), 0x1p126f);
      s = alpha * M * invC;
      cm = __fdiv_rn(448.0f, M);
    } else if (M != 0.0f) {  // far from 1: scaled by a power of two first, the energy from the result
      const int k = 1 - exponent_of(M);
#pragma unroll
      for (int i = 0; i < N; ++i) p1[i] = scale2(p1[i], k);
      const float Mk = scale2(M, k);
      const float sw = group_sum<L>(sum_squares<N>(p1));
      alpha = fminf(fmaxf(scale2((float)kB * __builtin_amdgcn_rsqf(sw), k), 0x1p-126f), 0x1p126f);
      s = scale2(alpha * Mk, -k) * invC;
      cm = __fdiv_rn(448.0f, Mk);
    }
    cm *= lane_sign<L>(j);
    constexpr int MADE = L == 4 ? 0 : GT == kGradCodes ? 2 : 1;  // the order after this transform
#pragma unroll
    for (int k = 0; k < NQ / 4; ++k) {
      uint32_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float *v = &p1[16 * k + 4 * i];
        d[i] = pack_fp8x4(fmaf(v[0], cm, 0.0f), fmaf(v[1], cm, 0.0f), fmaf(v[2], cm, 0.0f),
                          fmaf(v[3], cm, 0.0f));
      }
      const u32x4 c = quads_to_chunks<MADE>(d, j);
      if (bw * B < left)
        st_stream(c, (u32x4 *)((uint8_t *)e.copy + base + bw * B + 16 * L * k + 16 * chunk_of<L>(j)));
    }
    if (bw * B < left) {
      if (j == 0) {
        e.copy_alpha[base / B + bw] = alpha;
        e.copy_scale[base / B + bw] = s;
      }
    }
  }
}

}  // namespace tfp8

using namespace tfp8;

namespace {

constexpr int32_t kMostTensors = 1 << 24;

bool block_ok(int32_t b) { return b == 64 || b == 128 || b == 256 || b == 512; }

tfp8_status check_gradient(const tfp8_gradient &g, int32_t block) {
  if (g.n < 0 || g.n > TFP8_MAX_N) return TFP8_E_SIZE;
  if (g.dtype != TFP8_BF16 && g.dtype != TFP8_F32 && g.dtype != TFP8_CODES) return TFP8_E_DTYPE;
  if (g.dtype == TFP8_CODES && g.n % block != 0) return TFP8_E_SIZE;
  if (g.n == 0) return TFP8_OK;
  if (!g.data || (g.dtype == TFP8_CODES && (!g.alpha || !g.scale))) return TFP8_E_NULL;
  if (!aligned(g.data, 16) ||
      (g.dtype == TFP8_CODES && (!aligned(g.alpha, 4) || !aligned(g.scale, 4))))
    return TFP8_E_ALIGN;
  return TFP8_OK;
}

int64_t bytes_of(int64_t n, int64_t dtype) {
  return n * (dtype == TFP8_F32 ? 4 : dtype == TFP8_BF16 ? 2 : 1);
}

// Ranges of memory that a call reads and writes; whether one that is written meets another.
struct Spans {
  struct Span {
    uintptr_t lo, hi;
    bool written;
  };
  std::vector<Span> all;
  void add(const void *p, int64_t bytes, bool written) {
    if (bytes > 0) all.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
  }
  bool meet() {
    const auto before = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(all.begin(), all.end(), before)) std::sort(all.begin(), all.end(), before);
    uintptr_t any = 0, written = 0;  // where what came before ends
    for (const Span &s : all) {
      if (s.lo < written || (s.written && s.lo < any)) return true;
      any = std::max(any, s.hi);
      if (s.written) written = std::max(written, s.hi);
    }
    return false;
  }
};

int shift_of(int32_t block) { return block == 64 ? 6 : block == 128 ? 7 : block == 256 ? 8 : 9; }

// A tensor is handed to launches in pieces of at most this many elements, a launch of at most twice
// as many, so that its threads stay below 2^30.
constexpr int64_t kPiece = (int64_t)1 << 32;

struct StepLaunch {
  int32_t block;
  int32_t bits;
  bool p_f32;
  int grad;
  bool codes_out;
};

template <int B, bool PF32, int GT, int BITS, bool CC>
tfp8_status launch_step(const void *table, const StepArgs &a, unsigned grid, hipStream_t st) {
  constexpr bool ROT = GT == kGradCodes || CC;
  return launch(k_adamw<B, PF32, GT, BITS, CC>, grid, kThreads, st,
                *(const StepTable<ROT> *)table, a);
}

template <bool PF32, int GT, bool CC>
tfp8_status launch_step(const StepLaunch &l, const void *table, const StepArgs &a, unsigned grid,
                        hipStream_t st) {
  constexpr bool ROT = GT == kGradCodes || CC;
  if (l.bits == 32 && !ROT)  // no blocks at all
    return launch_step<128, PF32, GT, 32, CC>(table, a, grid, st);
#define TFP8_CASE(BB)                                                                     \
  case BB:                                                                                \
    if constexpr (ROT)                                                                    \
      if (l.bits == 32) return launch_step<BB, PF32, GT, 32, CC>(table, a, grid, st);     \
    return launch_step<BB, PF32, GT, 8, CC>(table, a, grid, st);
  switch (l.block) {
    TFP8_CASE(64)
    TFP8_CASE(128)
    TFP8_CASE(256)
    TFP8_CASE(512)
  }
#undef TFP8_CASE
  return TFP8_E_BLOCK;
}

template <bool PF32>
tfp8_status launch_step(const StepLaunch &l, const void *table, const StepArgs &a, unsigned grid,
                        hipStream_t st) {
  switch (l.grad) {
    case kGradBf16:
      return l.codes_out ? launch_step<PF32, kGradBf16, true>(l, table, a, grid, st)
                         : launch_step<PF32, kGradBf16, false>(l, table, a, grid, st);
    case kGradF32:
      return l.codes_out ? launch_step<PF32, kGradF32, true>(l, table, a, grid, st)
                         : launch_step<PF32, kGradF32, false>(l, table, a, grid, st);
    default:
      return l.codes_out ? launch_step<PF32, kGradCodes, true>(l, table, a, grid, st)
                         : launch_step<PF32, kGradCodes, false>(l, table, a, grid, st);
  }
}

// All tensors of one kind, a table at a time.
template <bool ROT>
tfp8_status launch_kind(const StepLaunch &l, const tfp8_adamw_tensor *tensors, int32_t count,
                        StepArgs a, hipStream_t st) {
  constexpr int NQ = 4;
  const int64_t tile = ROT ? 64 / lanes_per_block(l.block) * (int64_t)l.block : 64 * 4 * NQ;
  const int64_t per = tile * (kThreads / 64);  // elements a workgroup
  StepTable<ROT> t;
  memset(&t, 0, sizeof t);
  int used = 0;
  int64_t groups = 0;
  const auto flush = [&]() -> tfp8_status {
    if (!used) return TFP8_OK;
    a.count = used;
    const unsigned grid = (unsigned)groups;
    used = 0;
    groups = 0;
    return l.p_f32 ? launch_step<true>(l, &t, a, grid, st) : launch_step<false>(l, &t, a, grid, st);
  };
  for (int32_t i = 0; i < count; ++i) {
    const tfp8_adamw_tensor &x = tensors[i];
    if (x.grad.n == 0 || (x.param_dtype == TFP8_F32) != l.p_f32 || x.grad.dtype != l.grad ||
        (x.copy_dtype == TFP8_CODES) != l.codes_out)
      continue;
    for (int64_t at = 0; at < x.grad.n; at += kPiece) {
      const int64_t n = std::min(kPiece, x.grad.n - at), more = (n + per - 1) / per;
      if (used == StepTable<ROT>::kMost || (used && groups + more > 2 * kPiece / per)) {
        const tfp8_status s = flush();
        if (s != TFP8_OK) return s;
      }
      StepEntry<ROT> &e = t.e[used++];
      e.param = (char *)x.param + bytes_of(at, x.param_dtype);
      e.grad = (const char *)x.grad.data + bytes_of(at, x.grad.dtype);
      e.copy = x.copy_dtype == TFP8_NONE ? nullptr : (char *)x.copy + bytes_of(at, x.copy_dtype);
      e.n = n;
      e.start = x.start + at;
      e.first = groups;
      if constexpr (ROT) {
        const int64_t b = at / l.block;
        e.grad_alpha = x.grad.alpha ? x.grad.alpha + b : nullptr;
        e.grad_scale = x.grad.scale ? x.grad.scale + b : nullptr;
        e.copy_alpha = x.copy_alpha ? x.copy_alpha + b : nullptr;
        e.copy_scale = x.copy_scale ? x.copy_scale + b : nullptr;
      }
      groups += more;
    }
  }
  return flush();
}

tfp8_status grad_norm(const tfp8_gradient *grads, int32_t count, int32_t block, float max_norm,
                      void *workspace, int64_t workspace_bytes, float *norm, float *scale,
                      void *stream) {
  if (!block_ok(block)) return TFP8_E_BLOCK;
  if (count < 0 || count > kMostTensors) return TFP8_E_SIZE;
  if (!(max_norm > 0.0f)) return TFP8_E_ARG;
  if (!workspace || !norm || !scale || (count > 0 && !grads)) return TFP8_E_NULL;
  if (!aligned(workspace, 8) || !aligned(norm, 4) || !aligned(scale, 4)) return TFP8_E_ALIGN;
  const int64_t need = tfp8_grad_norm_workspace(count);
  if (workspace_bytes < need) return TFP8_E_SIZE;
  Spans spans;
  spans.all.reserve((size_t)count + 3);
  for (int32_t i = 0; i < count; ++i) {
    const tfp8_gradient &g = grads[i];
    const tfp8_status s = check_gradient(g, block);
    if (s != TFP8_OK) return s;
    spans.add(g.data, bytes_of(g.n, g.dtype), false);
    if (g.dtype == TFP8_CODES) {
      spans.add(g.alpha, g.n / block * 4, false);
      spans.add(g.scale, g.n / block * 4, false);
    }
  }
  spans.add(workspace, need, true);
  spans.add(norm, 4, true);
  spans.add(scale, 4, true);
  if (spans.meet()) return TFP8_E_ARG;
  hipStream_t st = (hipStream_t)stream;
  double *partial = (double *)workspace;
  int64_t parts = 0;
  NormTable t;
  memset(&t, 0, sizeof t);
  t.block_shift = shift_of(block);
  for (int32_t i = 0; i < count; ++i) {
    const tfp8_gradient &g = grads[i];
    if (g.n > 0) {
      NormEntry &e = t.e[t.count++];
      e = NormEntry{g.data, g.alpha, g.scale, g.n, t.units, g.dtype};
      t.units += (g.n + unit_elements(g.dtype) - 1) / unit_elements(g.dtype);
    }
    if (t.count == kNormTensors || (i == count - 1 && t.count > 0)) {
      const int64_t grid = std::min<int64_t>(t.units, kNormGrid);
      const tfp8_status s = launch(k_norm, (unsigned)grid, kThreads, st, t, partial + parts);
      if (s != TFP8_OK) return s;
      parts += grid;
      t.count = 0;
      t.units = 0;
    }
  }
  return launch(k_norm_finish, 1, kThreads, st, partial, parts, max_norm, norm, scale);
}

bool finite(double x) { return x - x == 0.0; }

tfp8_status adamw(const tfp8_adamw_tensor *tensors, int32_t count, int32_t block, int32_t bits,
                  const void *m, const float *m_scale, const void *v, const float *v_scale,
                  void *m_out, float *m_scale_out, void *v_out, float *v_scale_out,
                  int64_t state_n, const tfp8_adamw_options *o, void *stream) {
  if (!block_ok(block)) return TFP8_E_BLOCK;
  if (count < 0 || count > kMostTensors || state_n < 0 || state_n > TFP8_MAX_N) return TFP8_E_SIZE;
  if (!o) return TFP8_E_NULL;
  if (bits != 8 && bits != 32) return TFP8_E_ARG;
  if (!(o->beta1 >= 0.0 && o->beta1 < 1.0 && o->beta2 >= 0.0 && o->beta2 < 1.0) ||
      !((float)o->eps >= 0x1p-126f) || !finite(o->eps) || !finite(o->lr) ||
      !finite(o->weight_decay) || o->step < 1)
    return TFP8_E_ARG;
  if ((o->lr_dev || o->step_dev) && !o->workspace) return TFP8_E_NULL;
  if (!aligned(o->lr_dev, 4) || !aligned(o->step_dev, 8) || !aligned(o->grad_scale, 4) ||
      !aligned(o->workspace, 8))
    return TFP8_E_ALIGN;
  if (count > 0 && !tensors) return TFP8_E_NULL;
  int64_t end = 0;
  bool any = false;
  Spans spans;
  spans.all.reserve((size_t)count * 4 + 8);
  bool kinds[2][3][2] = {};
  for (int32_t i = 0; i < count; ++i) {
    const tfp8_adamw_tensor &x = tensors[i];
    const tfp8_status s = check_gradient(x.grad, block);
    if (s != TFP8_OK) return s;
    if (x.param_dtype != TFP8_BF16 && x.param_dtype != TFP8_F32) return TFP8_E_DTYPE;
    if (x.copy_dtype != TFP8_NONE && x.copy_dtype != TFP8_BF16 && x.copy_dtype != TFP8_CODES)
      return TFP8_E_DTYPE;
    const bool codes = x.copy_dtype == TFP8_CODES;
    const int64_t n = x.grad.n;
    if (x.start < 0 || x.start > TFP8_MAX_N || x.start % block != 0 || (codes && n % block != 0))
      return TFP8_E_SIZE;
    if (n == 0) continue;
    if (x.start < end) return TFP8_E_ARG;
    end = (x.start + n + block - 1) / block * block;
    if (end > state_n) return TFP8_E_ARG;  // its last block has a scale, too
    if (!x.param || (x.copy_dtype != TFP8_NONE && !x.copy) ||
        (codes && (!x.copy_alpha || !x.copy_scale)))
      return TFP8_E_NULL;
    if (!aligned(x.param, 16) || (x.copy_dtype != TFP8_NONE && !aligned(x.copy, 16)) ||
        (codes && (!aligned(x.copy_alpha, 4) || !aligned(x.copy_scale, 4))))
      return TFP8_E_ALIGN;
    any = true;
    kinds[x.param_dtype == TFP8_F32][x.grad.dtype][codes] = true;
    spans.add(x.param, bytes_of(n, x.param_dtype), true);
    spans.add(x.grad.data, bytes_of(n, x.grad.dtype), false);
    if (x.grad.dtype == TFP8_CODES) {
      spans.add(x.grad.alpha, n / block * 4, false);
      spans.add(x.grad.scale, n / block * 4, false);
    }
    if (x.copy_dtype != TFP8_NONE) spans.add(x.copy, bytes_of(n, x.copy_dtype), true);
    if (codes) {
      spans.add(x.copy_alpha, n / block * 4, true);
      spans.add(x.copy_scale, n / block * 4, true);
    }
  }
  if (!any) return TFP8_OK;
  // each of the four states: where it comes from, where it goes to, its bytes and alignment
  const int64_t each = bits == 8 ? state_n : state_n * 4, scales = state_n / block * 4;
  const struct {
    const void *in, *out;
    int64_t bytes;
    uintptr_t align;
  } states[4] = {{m, m_out, each, 16},
                 {v, v_out, each, 16},
                 {m_scale, m_scale_out, scales, 4},
                 {v_scale, v_scale_out, scales, 4}};
  for (int i = 0; i < (bits == 8 ? 4 : 2); ++i)
    if (!states[i].in || !states[i].out) return TFP8_E_NULL;
  for (int i = 0; i < (bits == 8 ? 4 : 2); ++i) {
    if (!aligned(states[i].in, states[i].align) || !aligned(states[i].out, states[i].align))
      return TFP8_E_ALIGN;
    if (states[i].in != states[i].out) spans.add(states[i].in, states[i].bytes, false);
    spans.add(states[i].out, states[i].bytes, true);
  }
  if (o->lr_dev) spans.add(o->lr_dev, 4, false);
  if (o->step_dev) spans.add(o->step_dev, 8, false);
  if (o->grad_scale) spans.add(o->grad_scale, 4, false);
  const bool on_device = o->lr_dev || o->step_dev;
  if (on_device) spans.add(o->workspace, 32, true);
  if (spans.meet()) return TFP8_E_ARG;

  StepArgs a{};
  a.m = m;
  a.v = v;
  a.m_scale = m_scale;
  a.v_scale = v_scale;
  a.m_out = m_out;
  a.v_out = v_out;
  a.m_scale_out = m_scale_out;
  a.v_scale_out = v_scale_out;
  a.grad_scale = o->grad_scale;
  a.beta1 = (float)o->beta1;
  a.rest1 = (float)(1.0 - o->beta1);
  a.beta2 = (float)o->beta2;
  a.root2 = (float)sqrt(o->beta2);
  a.root_rest2 = (float)sqrt(1.0 - o->beta2);
  a.eps = (float)o->eps;
  hipStream_t st = (hipStream_t)stream;
  if (on_device) {
    a.factors = (const Factors *)o->workspace;
    const tfp8_status s =
        launch(k_adamw_factors, 1, 64, st, o->lr, o->beta1, o->beta2, o->weight_decay, o->step,
               o->seed, o->lr_dev, o->step_dev, (Factors *)o->workspace);
    if (s != TFP8_OK) return s;
  } else {
    a.f = factors_of(o->lr, o->beta1, o->beta2, o->weight_decay, o->step, o->seed);
  }
  for (int p = 0; p < 2; ++p)
    for (int g = 0; g < 3; ++g)
      for (int c = 0; c < 2; ++c) {
        if (!kinds[p][g][c]) continue;
        const StepLaunch l{block, bits, p == 1, g, c == 1};
        const tfp8_status s = g == kGradCodes || c == 1 ? launch_kind<true>(l, tensors, count, a, st)
                                                        : launch_kind<false>(l, tensors, count, a, st);
        if (s != TFP8_OK) return s;
      }
  return TFP8_OK;
}

}  // namespace

extern "C" {

int64_t tfp8_grad_norm_workspace(int32_t count) {
  if (count < 0 || count > kMostTensors) return 0;
  const int64_t launches = ((int64_t)count + kNormTensors - 1) / kNormTensors;
  return 8 * kNormGrid * (launches > 0 ? launches : 1);
}

// The lists of memory ranges are the only host memory that these two take; a call that gets none
// launches nothing.
tfp8_status tfp8_grad_norm(const tfp8_gradient *grads, int32_t count, int32_t block, float max_norm,
                           void *workspace, int64_t workspace_bytes, float *norm, float *scale,
                           void *stream) {
  try {
    return grad_norm(grads, count, block, max_norm, workspace, workspace_bytes, norm, scale, stream);
  } catch (const std::bad_alloc &) {
    return TFP8_E_SIZE;
  }
}

tfp8_status tfp8_adamw(const tfp8_adamw_tensor *tensors, int32_t count, int32_t block, int32_t bits,
                       const void *m, const float *m_scale, const void *v, const float *v_scale,
                       void *m_out, float *m_scale_out, void *v_out, float *v_scale_out,
                       int64_t state_n, const tfp8_adamw_options *options, void *stream) {
  try {
    return adamw(tensors, count, block, bits, m, m_scale, v, v_scale, m_out, m_scale_out, v_out,
                 v_scale_out, state_n, options, stream);
  } catch (const std::bad_alloc &) {
    return TFP8_E_SIZE;
  }
}

}  // extern "C"
