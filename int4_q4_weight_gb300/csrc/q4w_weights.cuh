// Weights of logits as integers, for masses whose sums have no order and whose borders
// fall on the side that the definition says: 2^-t, t = (M - z) log2(e) / T, cut into
// n = floor(8 t), an eighth of an octave, and a 28-bit mantissa of the rest.
#pragma once

#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "q4w_device.cuh"
#include "q4w_kv.cuh"

namespace q4w {
namespace sample {

constexpr int kBins = 1024;         // eighths of 128 octaves
typedef unsigned long long u64;

// What turns a logit of this row into a weight.
struct Scale {
  float top;       // M, the largest finite number for an infinite maximum
  float ch, cl;    // 8 log2(e) / T in two pieces
  u64 minp;        // min_p in units of 2^-59, 0: off
};

__device__ __forceinline__ Scale make_scale(float top, float temp, float min_p) {
  Scale s;
  s.top = fminf(top, CUDART_MAX_NORMAL_F);
  // 8 log2(e) = h + l; the quotient's remainder is exact
  const float h = 11.541560173034668f, l = 1.540770427e-07f;
  const float t = fmaxf(temp, 1e-36f);
  s.ch = h / t;
  const float r = fmaf(-s.ch, t, h) + l;
  s.cl = r / t;
  if (!(s.ch < 1e38f) || temp == CUDART_INF_F) s.cl = 0.f;
  const float m = fminf(min_p, 1.f);
  s.minp = min_p > 0.f ? max((u64)(m * 576460752303423488.f), 1ull) : 0ull;   // a power of two times m: exact
  return s;
}

// A logit as the passes see it: +inf becomes the largest finite number, a NaN
// stays one and fails every comparison.
__device__ __forceinline__ float capped(const Scale& s, float z) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(s.top));
  return r;
}
// 8 t, rounded: it only cuts the weights into bins, the same way everywhere.
// Not below kBins (or NaN): the weight is below 2^-128 and never counts.
__device__ __forceinline__ float eighths(const Scale& s, float z) { return (s.top - z) * s.ch; }

// floor(q) for 0 <= q < 2^22, as a number and as an integer, without the
// conversion unit (a quarter of the rate of an addition or less).
__device__ __forceinline__ int whole(float q, float* n) {
  const float t = __fadd_rd(q, 8388608.f);
  *n = t - 8388608.f;
  return __float_as_int(t) & 0x7fffff;
}

// 28-bit mantissa of the weight inside its bin n: 2^-(t - n/8), in (0.9, 1] * 2^28.
__device__ __forceinline__ uint32_t mantissa(const Scale& s, float z, float q, float n) {
  const float d = s.top - z, bb = d - s.top;
  const float dl = (s.top - (d - bb)) - (z + bb);           // the exact difference is d + dl
  const float e = fmaf(d, s.ch, -q) + fmaf(d, s.cl, dl * s.ch);
  const float f = (q - n) + e;
  // (2^(-f/8) - 1) 2^28 on [0, 1]: the series of exp(-f ln 2 / 8); the next term is below 2^-9
  float g = 1.577321512e-01f;
  g = fmaf(g, f, -1.092285083e+01f);
  g = fmaf(g, f, 6.303337092e+02f);
  g = fmaf(g, f, -2.910013812e+04f);
  g = fmaf(g, f, 1.007582999e+06f);
  g = fmaf(g, f, -2.325815994e+07f);
  return (uint32_t)((1 << 28) + __float2int_rn(g * f));
}

// 2^(-j/8) * 2^31, rounded; the kernel keeps a copy in shared memory (lanes that
// ask for different entries of constant memory wait for one another).
static __device__ __constant__ uint32_t kEighth[8] = {2147483648u, 1969251188u, 1805811301u, 1655936265u,
                                               1518500250u, 1392470869u, 1276901417u, 1170923762u};

__device__ __forceinline__ u64 shift_right(u64 x, int by) {   // 0 from 64 on
  u64 r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(x), "r"(by));
  return r;
}
// The weight in units of 2^-42 (2^-59 before the shift), cut off.
__device__ __forceinline__ u64 weight_of(const uint32_t* eighth, uint32_t mant, int n) {
  return shift_right((u64)mant * eighth[n & 7], 17 + (n >> 3));
}
// Of any logit, a NaN among them, without a branch: the elements of a thread are
// computed side by side.  Beyond the bins the shift leaves nothing.
__device__ __forceinline__ u64 weight(const uint32_t* eighth, const Scale& s, float z) {
  const float q = fminf(eighths(s, z), (float)kBins - 1.f);
  float nf;
  const int n = whole(q, &nf);
  return weight_of(eighth, mantissa(s, z, q, nf), n);
}

// Two weights' parts at once, in packed fp32: bit for bit what eighths(), whole() and mantissa()
// give (every step rounds alike; differences are formed with the signs turned, which rounds alike
// too).  Some 25 instructions a weight for 42.
struct Pair {
  uint32_t mant[2];
  int n[2];
};
__device__ __forceinline__ f2_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ Pair mantissas(const Scale& s, float z0, float z1) {
  const f2_t minus = f2_both(-1.f), top = f2_both(s.top), ch = f2_both(s.ch);
  auto sub = [&](f2_t a, f2_t b) { return f2_fma(b, minus, a); };
  const f2_t z = f2_pack(capped(s, z0), capped(s, z1));
  const f2_t nd = f2_add(z, f2_both(-s.top));   // -(top - z)
  float q0, q1;
  f2_unpack(f2_mul(nd, f2_both(-s.ch)), q0, q1);
  const f2_t q = f2_pack(fminf(q0, (float)kBins - 1.f), fminf(q1, (float)kBins - 1.f));
  f2_t t;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(t) : "l"(q), "l"(f2_both(8388608.f)));
  const f2_t n = f2_add(t, f2_both(-8388608.f));
  const f2_t nb = f2_add(nd, top);
  const f2_t dl = sub(sub(top, sub(nb, nd)), sub(z, nb));
  const f2_t e = sub(f2_fma(nd, f2_both(-s.cl), f2_mul(dl, ch)), f2_fma(nd, ch, q));
  const f2_t f = f2_add(sub(q, n), e);
  f2_t g = f2_both(1.577321512e-01f);
  g = f2_fma(g, f, f2_both(-1.092285083e+01f));
  g = f2_fma(g, f, f2_both(6.303337092e+02f));
  g = f2_fma(g, f, f2_both(-2.910013812e+04f));
  g = f2_fma(g, f, f2_both(1.007582999e+06f));
  g = f2_fma(g, f, f2_both(-2.325815994e+07f));
  float g0, g1, t0, t1;
  f2_unpack(f2_mul(g, f), g0, g1);
  f2_unpack(t, t0, t1);
  return {{(uint32_t)((1 << 28) + __float2int_rn(g0)), (uint32_t)((1 << 28) + __float2int_rn(g1))},
          {__float_as_int(t0) & 0x7fffff, __float_as_int(t1) & 0x7fffff}};
}

__device__ __forceinline__ bool passes_minp(const uint32_t* eighth, const Scale& s, float z) {
  const float q = fminf(eighths(s, z), (float)kBins - 1.f);
  float nf;
  const int n = whole(q, &nf);
  return shift_right((u64)mantissa(s, z, q, nf) * eighth[n & 7], n >> 3) >= s.minp;
}

// floor (or ceiling) of m * f for 0 <= f < 1, exactly.
static __device__ __noinline__ u64 times(u64 m, float f, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const u64 mant = ex ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - max(ex, 1);                 // f = mant * 2^-sh, sh >= 24
  const u64 lo = m * mant, hi = __umul64hi(m, mant);
  u64 q, rest;
  if (sh < 64) q = (lo >> sh) | (hi << (64 - sh)), rest = lo << (64 - sh);
  else if (sh == 64) q = hi, rest = lo;
  else if (sh < 128) q = hi >> (sh - 64), rest = lo | (hi << (128 - sh));
  else q = 0, rest = lo | hi;
  return q + (up && rest ? 1 : 0);
}

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}

}  // namespace sample
}  // namespace q4w
