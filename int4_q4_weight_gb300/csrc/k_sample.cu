// Sampling a token per row of logits: temperature, top-k, top-p and min-p,
// from a given random number.
//
// With M = max z and w_i = 2^-t_i, t_i = (M - z_i) log2(e) / T:
//   S_k  the k largest z (ties: lower index first),
//   S_p  the shortest prefix of S_k in that order whose mass reaches
//        p mass(S_k),
//   S    those of S_p with w_i >= min_p,
//   token = the first index, in vocabulary order, whose running mass in S
//        exceeds u mass(S);  logprob = ln(w_token / mass(S)).
// All three sets are prefixes of one order, so S is given by a threshold
// (the key of a logit and how many of its ties, lowest index first) and the
// min-p test.  Nothing is sorted over the vocabulary.
//
// Arithmetic.  A token that lies next to a border has to fall on the side
// that the definition says, and a border is a sum of up to 2^20 weights, so
// fp32 sums of expf would be too coarse: masses are integers.  8 t is formed as
// an fp32 pair (the difference exactly, 8 log2(e)/T in two pieces), cut into
// n = floor(8 t), an eighth of an octave, and the rest f in [0, 1], which goes
// through a degree-6 polynomial of 2^(-f/8) to a 28-bit mantissa; the weight is
// mantissa * 2^(-(n mod 8)/8) * 2^-(n div 8), cut off to units of 2^-42.
// Integer sums have no order, so atomics and cluster reductions give the same
// bits on every run.  A weight is off by up to 2^-26 of itself (2^-28.8 in the
// root mean square: the polynomial in fp32 is most of it), and cut downwards by
// less than a unit: a sum of n weights is up to n 2^-42 of the largest too small, and
// nothing is left of a weight below 2^-42.  The log probability is therefore formed
// from the chosen logit, ln of the mass alone from the integers; and u = 0, which asks
// for the first of S however small its weight, goes by the members of S instead.
// Products of a mass with top_p or u are formed exactly in 128 bits (fp64 runs
// at a sixtieth of the fp32 rate: one logarithm per row is all of it).
//
// Work.  A cluster of CTAs takes a row, each an index range of it:
//   A  the maximum (greedy rows: then its lowest index);
//   B  a histogram of n over the row (1024 bins: 128 octaves), which bounds
//      the last bin that S can reach;
//   C  few candidates (<= 2048) up to that bin: they are gathered into the
//      leader CTA, ranked, cut and sampled there;
//   D  many: the bin that holds a border is refined by histograms of the
//      order-preserving integer key (1024 sub-bins a level) until the
//      threshold is a single key; then masses of 128-index segments, a scan of
//      them, and the one segment that holds the target.
//   E  top-p without top-k goes by the mass of the whole row.  Instead of B to D:
//      a histogram of short weights bounds where the border lies; when at most
//      2048 elements lie there, one pass forms the exact mass of the row and of
//      the segments above them, and the leader sorts those few and cuts.
//      (Exact weights are formed once, not twice, and a bin is one atomic
//      addition, not three: 8 rows of 262144, top-p 0.9: 42 us, by B to D 53;
//      192 rows 300 against 388.  The code costs top-64 of a few rows 1.3 us.)
// The row is read from HBM once; the later passes find it in registers (few rows)
// or in L2.
#include <math_constants.h>

#include "q4w_device.cuh"
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"
#include "q4w_tc.cuh"

namespace q4w {
namespace sample {

constexpr int kThr = 512;
constexpr int kWarpsS = kThr / 32;
constexpr int kBins = 1024;
static_assert(kBins == 2 * kThr, "a thread has two bins of a merged histogram");
constexpr int kCap = 2048;          // candidates that the leader takes
constexpr int kCount = 256;         // up to here they are ranked by counting, else sorted
constexpr int kSortFew = 1024;      // around the border of top-p: up to here they are sorted, else the range refined
constexpr int kSeg = 128;           // indices per segment of the final pass
constexpr int kMaxSegs = 1024;      // segments of a CTA: 2^17 indices, so a 32-bit bin never overflows
constexpr int kKeep = 64;           // indices a thread may keep in registers
typedef unsigned long long u64;

struct Params {
  const void* z;               // [rows][V]
  long long stride;            // elements
  const float* u;
  const float* temperature;    // NULL: 1
  const int32_t* top_k;        // NULL or <= 0: off
  const float* top_p;          // NULL or >= 1: off
  const float* min_p;          // NULL or <= 0: off
  int32_t* token;
  float* logprob;              // NULL: not written
  int V;
  int range;                   // indices per CTA of the cluster, a multiple of kSeg
  int rows;
  int order;                   // more rows than run at once: costly ones first
};

// Order-preserving integer of a logit: larger logit, larger key; 0 and -0 tie.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// The upper end of a range of keys as a logit.  The key below 0's is -0's, which no
// logit has, and a comparison with -0 would let 0 in.
__device__ __forceinline__ float logit_below(uint32_t k) { return logit_of(k == 0x7fffffffu ? k - 1 : k); }

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
__device__ __constant__ uint32_t kEighth[8] = {2147483648u, 1969251188u, 1805811301u, 1655936265u,
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
__device__ __forceinline__ bool passes_minp(const uint32_t* eighth, const Scale& s, float z) {
  const float q = fminf(eighths(s, z), (float)kBins - 1.f);
  float nf;
  const int n = whole(q, &nf);
  return shift_right((u64)mantissa(s, z, q, nf) * eighth[n & 7], n >> 3) >= s.minp;
}

// floor (or ceiling) of m * f for 0 <= f < 1, exactly.
__device__ __noinline__ u64 times(u64 m, float f, bool up) {
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

// ln of the chosen logit's share of the mass: from the logit, not from its weight in
// whole units, of which a small one keeps few digits or none.
__device__ __noinline__ float log_prob(const Params& p, int row, float top, float v, u64 mass) {
  const float t = p.temperature ? fmaxf(p.temperature[row], 1e-36f) : 1.f;
  return (float)(((double)v - (double)top) / (double)t - log((double)mass * 2.2737367544323206e-13));
}

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}

// E consecutive logits from index i on, a multiple of E; NaN behind i1 (a NaN is
// neither a maximum nor below any bound).  vec: the row begins on a 16-byte
// boundary.
template <typename T, int E>
__device__ __forceinline__ void load_logits(const T* row, int i, int i1, bool vec, float (&v)[E]) {
  if (vec && i + E <= i1) {
    T e[E];
    if constexpr (sizeof(e) == 16) *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(row + i);
    else *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(row + i);
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = as_float(e[k]);
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = i + k < i1 ? as_float(row[i + k]) : CUDART_NAN_F;
  }
}

// A CTA's part [i0, i1) of the row, i0 a multiple of kSeg.  KEEP: the part has at
// most kKeep indices a thread, which stay in registers from the first pass on.
template <typename T, bool KEEP>
struct Part {
  static constexpr int E = 16 / sizeof(T), kVecs = kKeep / E, step = E * kThr;
  const T* row;
  int i0, i1;
  bool vec;
  float v[KEEP ? kKeep : 1];

  __device__ __forceinline__ void load() {
    if constexpr (KEEP) {
#pragma unroll
      for (int x = 0; x < kVecs; ++x) {
        float t[E];
        load_logits<T, E>(row, i0 + E * (int)threadIdx.x + x * step, i1, vec, t);
#pragma unroll
        for (int k = 0; k < E; ++k) v[x * E + k] = t[k];
      }
    }
  }
  // Calls f(logit, index) for every index, and with NaNs behind them, in no
  // order: short bodies.
  template <typename F>
  __device__ __forceinline__ void light(F f) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int x = 0; x < kVecs; ++x)
#pragma unroll
        for (int k = 0; k < E; ++k) f(v[x * E + k], i0 + E * (int)threadIdx.x + x * step + k);
    } else {
      constexpr int U = sizeof(T) == 4 ? 4 : 2;   // loads in flight
      int i = i0 + E * (int)threadIdx.x;
      if (vec) {
#pragma unroll 1
        for (; i + (U - 1) * step + E <= i1; i += U * step) {
          float t[U][E];
#pragma unroll
          for (int x = 0; x < U; ++x) load_logits<T, E>(row, i + x * step, 0x7fffffff, true, t[x]);
#pragma unroll
          for (int x = 0; x < U; ++x)
#pragma unroll
            for (int k = 0; k < E; ++k) f(t[x][k], i + x * step + k);
        }
      }
#pragma unroll 1
      for (; i < i1; i += step) {
        float t[E];
        load_logits<T, E>(row, i, i1, vec, t);
#pragma unroll
        for (int k = 0; k < E; ++k) f(t[k], i + k);
      }
    }
  }
  // Calls act(logit, index) for the few logits that pred holds for: the test is
  // expanded for every element, the body exists once.
  template <typename P, typename A>
  __device__ __forceinline__ void rare(P pred, A act) const {
    int base = 0;
    uint32_t hits = 0;   // of 32 elements
    auto take = [&](int first) {
      while (hits) {
        const int b = first + __ffs(hits) - 1;
        hits &= hits - 1;
        const int i = base + b / E * step + b % E;
        act(as_float(row[i]), i);
      }
    };
    base = i0 + E * (int)threadIdx.x;
    if constexpr (KEEP) {
      uint32_t all[kKeep / 32];
#pragma unroll
      for (int h = 0; h < kKeep / 32; ++h) {
        all[h] = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) all[h] |= pred(v[32 * h + k]) ? 1u << k : 0u;
      }
#pragma unroll 1
      for (int h = 0; h < kKeep / 32; ++h) {
        hits = h == 0 ? all[0] : all[1];
        take(32 * h);
      }
      static_assert(kKeep == 64, "two words of hits");
    } else {
#pragma unroll 1
      for (; base < i1; base += 32 / E * step) {
        hits = 0;
#pragma unroll
        for (int x = 0; x < 32 / E; ++x) {
          float t[E];
          load_logits<T, E>(row, base + x * step, i1, vec, t);
#pragma unroll
          for (int k = 0; k < E; ++k) hits |= pred(t[k]) ? 1u << (x * E + k) : 0u;
        }
        take(0);
      }
    }
  }
  // The same as light() for long bodies, expanded for one load only, the next one
  // in flight meanwhile.
  template <typename F>
  __device__ __forceinline__ void heavy(F f) const {
    float next[E];
    load_logits<T, E>(row, i0 + E * (int)threadIdx.x, i1, vec, next);
#pragma unroll 1
    for (int i = i0 + E * (int)threadIdx.x; i < i1; i += step) {
      float t[E];
#pragma unroll
      for (int k = 0; k < E; ++k) t[k] = next[k];
      load_logits<T, E>(row, i + step, i1, vec, next);
#pragma unroll
      for (int k = 0; k < E; ++k) f(t[k], i + k);
    }
  }
};

__device__ __forceinline__ u64 ld_cluster_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  tc::cluster_arrive_release();
  tc::cluster_wait();
}

// Sum of a 64-bit value that every CTA has at `v`, and of those of the CTAs
// before this one: lane r asks CTA r.
__device__ __forceinline__ u64 cluster_sum(const u64* v, uint32_t rank, uint32_t ctas, u64* before) {
  const uint32_t lane = threadIdx.x & 31;
  u64 x = lane < ctas ? ld_cluster_u64(tc::cluster_addr(v, lane)) : 0ull, y = lane < rank ? x : 0ull;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  *before = __shfl_sync(0xffffffffu, y, 0);
  return __shfl_sync(0xffffffffu, x, 0);
}

struct Shared {
  uint32_t cnt[kBins], lo[kBins], hi[kBins];   // per bin: elements, sums of the mantissa's low 14 and high bits
  union {
    u64 list[kCap];                            // candidates: inverted key, index
    u64 seg[kMaxSegs];                         // masses of the segments
  };
  uint32_t tie[kMaxSegs];                      // elements equal to the threshold, per segment
  int row;                                     // of this cluster, where costly rows go first
  float top;                                   // this CTA's maximum
  int first;                                   // its first index that holds the row's
  u64 mine;                                    // this CTA's mass of S
  u64 ties;                                    // this CTA's elements equal to the threshold
  uint32_t n_list;
  u64 red[kWarpsS];
  uint32_t red32[kWarpsS];
  u64 scan_total;
  // a range of bins or keys that holds the border of top-p
  int j_lo, j_hi;
  u64 c_lo, c_hi, m_lo;
  // of the leader: the last kept element of its list, and how many are kept
  u64 last_kept;
  int n_kept;
  uint32_t eighth[8];
  // the crossing bin of a scan
  int cross_bin;
  uint32_t cross_cnt;
  u64 cross_mass;
};

template <typename V>
__device__ __forceinline__ V warp_incl(V v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// Inclusive scan over the CTA's threads; *total: the sum.
template <typename V>
__device__ __forceinline__ V block_incl(V v, V* red, V* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_incl(v);
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  V before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarpsS; ++w) {
    if (w < warp) before += red[w];
    sum += red[w];
  }
  *total = sum;
  return v + before;
}

// Ascending bitonic sort of n values in shared memory, n a power of two.  A
// warp's 32 pairs of a step lie in 64 neighbouring values when they are at most
// 32 apart, so only the wider steps need the whole CTA.
__device__ __noinline__ void bitonic(u64* v, int n) {
  __syncthreads();
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int p = threadIdx.x; p < n / 2; p += kThr) {
        const int i = p + (p & ~(j - 1)), x = i + j;
        const u64 a = v[i], b = v[x];
        if ((a > b) == ((i & k) == 0)) v[i] = b, v[x] = a;
      }
      if (j > 32 || (j == 1 && k >= 64)) __syncthreads(); else __syncwarp();
    }
  __syncthreads();
}

// Adds every CTA's histogram, in every CTA: bins 2 threadIdx.x and + 1.
__device__ __forceinline__ void merge_bins(Shared& sh, uint32_t ctas, bool masses, u64 (&cnt)[2], u64 (&mant)[2]) {
  cnt[0] = cnt[1] = mant[0] = mant[1] = 0;
#pragma unroll 8
  for (uint32_t r = 0; r < ctas; ++r) {
    const u64 c = ld_cluster_u64(tc::cluster_addr(&sh.cnt[2 * threadIdx.x], r));
    cnt[0] += (uint32_t)c, cnt[1] += c >> 32;
    if (masses) {
      const u64 l = ld_cluster_u64(tc::cluster_addr(&sh.lo[2 * threadIdx.x], r));
      const u64 h = ld_cluster_u64(tc::cluster_addr(&sh.hi[2 * threadIdx.x], r));
      mant[0] += (uint32_t)l + ((u64)(uint32_t)h << 14);
      mant[1] += (l >> 32) + ((h >> 32) << 14);
    }
  }
}

__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int i = threadIdx.x; i < kBins; i += kThr) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
}

__device__ __forceinline__ void add_to_bin(Shared& sh, int b, uint32_t mant) {
  atomicAdd(&sh.cnt[b], 1u);
  atomicAdd(&sh.lo[b], mant & 0x3fffu);
  atomicAdd(&sh.hi[b], mant >> 14);
}

// Mass of a bin whose elements' mantissas sum to m, in units of 2^-42.
__device__ __forceinline__ u64 bin_mass(const uint32_t* eighth, u64 m, int n) {
  // m < 2^49: in two pieces so that the product with the 32-bit factor fits
  const u64 e = eighth[n & 7];
  const u64 a = (m >> 24) * e, b = (m & 0xffffffu) * e;   // 2^59 scale: a << 24 + b
  const int sh = 17 + (n >> 3);
  if (sh > 80) return 0ull;
  return (sh >= 24 ? a >> (sh - 24) : a << (24 - sh)) + (sh < 60 ? b >> sh : 0ull);
}

// The smallest key in [-inf, top] whose logit `ok` holds for; it holds for the top
// and, once it holds, for everything above.  A 32-way search, the same in each warp.
template <typename F>
__device__ __forceinline__ uint32_t smallest_key(const Scale& s, F ok) {
  const int lane = threadIdx.x & 31;
  uint32_t a = key_of(-CUDART_INF_F), b = key_of(s.top);
  while (a < b) {
    const uint32_t span = b - a, part = span / 32 + 1;
    const uint32_t k = min(a + part * lane, b);
    const uint32_t yes = __ballot_sync(0xffffffffu, k == b || ok(logit_of(k)));
    const int f = yes ? __ffs(yes) - 1 : 32;   // the first that qualifies
    const uint32_t below = __shfl_sync(0xffffffffu, k, f > 0 ? f - 1 : 0), at = __shfl_sync(0xffffffffu, k, f & 31);
    if (yes) b = at;
    if (f > 0) a = below + 1;
  }
  return b;
}
__device__ __forceinline__ uint32_t first_key(const Scale& s, float edge) {   // of the bins before `edge`
  return smallest_key(s, [&](float v) { return eighths(s, v) < edge; });
}
__device__ __noinline__ uint32_t minp_key(const uint32_t* eighth, Scale s) {
  return smallest_key(s, [&](float v) { return passes_minp(eighth, s, v); });
}

// 2^(x / 8), to 22 bits.
__device__ __forceinline__ float ex2_eighth(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 0.125f));
  return r;
}

// Top-p over a whole row: a range of keys [*k_lo, *k_hi], at most kCap elements,
// that holds the border, from masses with error bounds.  False where kCap elements
// lie closer to the border than the bounds: many ties, or p next to 1.
//
// A weight enters with 14 to 16 bits, rounded (as many as the sum of a CTA's part
// leaves of 32), so that a bin is one atomic addition; its error, that of 8 t in
// fp32 and of ex2.approx are below eps of it.  The prefix masses are exact sums.
template <typename T, bool KEEP>
__device__ __forceinline__ bool narrow(const Part<T, KEEP>& part, Shared& sh, const Scale& s, float top_p, int range,
                                       uint32_t ctas, uint32_t* k_lo_out, uint32_t* k_hi_out) {
  const int lane = threadIdx.x & 31, b0 = 2 * threadIdx.x;
  const int bits = min(31 - (32 - __clz(range - 1)), 16);
  const float unit = (float)(1 << bits), eps = 0.6f / unit + 1.6e-5f;
  part.heavy([&](float v, int) {
    const float q = eighths(s, capped(s, v));
    if (q < (float)kBins) {
      float nf;
      const int n = whole(q, &nf);
      atomicAdd(&sh.cnt[n], __float_as_uint(fmaf(ex2_eighth(nf - q), unit, 8388608.f)) & 0x7fffffu);
    }
  });
  if (threadIdx.x == 0) sh.j_lo = sh.j_hi = kBins - 1;
  cluster_sync();
  u64 c[2], m[2], tot, all;
  merge_bins(sh, ctas, false, c, m);
  u64 w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) w[j] = bin_mass(sh.eighth, c[j] << (28 - bits), b0 + j);
  const u64 w_in = block_incl(w[0] + w[1], sh.red, &tot), c_in = block_incl(c[0] + c[1], sh.red, &all);
  // what the exact p mass(row) lies between; the cutting of weights to 2^-42 is below 2^-22 of the mass
  const float want = top_p * (float)tot, cut = 3e-7f * (float)tot;
  const float want_lo = want * (1.f - eps) - cut, want_hi = want * (1.f + eps) + cut;
  // the first bins where S_p may end and where it must have ended
  auto find = [&](bool lo0, bool lo1, bool hi0, bool hi1) {
    const int lo = __reduce_min_sync(0xffffffffu, lo0 ? b0 : lo1 ? b0 + 1 : kBins - 1);
    const int hi = __reduce_min_sync(0xffffffffu, hi0 ? b0 : hi1 ? b0 + 1 : kBins - 1);
    if (lane == 0) atomicMin(&sh.j_lo, lo), atomicMin(&sh.j_hi, hi);
    __syncthreads();
  };
  {
    const float w0 = (float)(w_in - w[1]), w1 = (float)w_in;
    find(w0 * (1.f + eps) >= want_lo, w1 * (1.f + eps) >= want_lo, w0 * (1.f - eps) >= want_hi, w1 * (1.f - eps) >= want_hi);
  }
  const int bin = sh.j_lo, bin_hi = sh.j_hi;
  if ((bin & ~1) == b0) sh.c_lo = bin & 1 ? c_in - c[1] : c_in - c[1] - c[0], sh.m_lo = bin & 1 ? w_in - w[1] : w_in - w[1] - w[0];
  if ((bin_hi & ~1) == b0) sh.c_hi = bin_hi & 1 ? c_in : c_in - c[1];
  __syncthreads();
  u64 inside = (u64)((float)(sh.c_hi - sh.c_lo) / (0.91f * unit)) + 1;   // at most: a weight is 0.917 units or more
  float m_lo = (float)sh.m_lo * (1.f - eps), m_hi = (float)sh.m_lo * (1.f + eps);   // the mass before the range
  uint32_t k_lo = first_key(s, (float)(bin_hi + 1)), k_hi = bin == 0 ? key_of(s.top) : first_key(s, (float)bin) - 1;
  // Three levels of 1024 take up to 2^30 off the range, less where the bounds are wide;
  // what is still too many then (a flat row's range is near 2^32 keys) goes the way of
  // B to D.  (A level takes 4 us of a few rows, the sorting of 2048 elements 11 us more
  // than that of 1024.)
  for (int level = 0; inside > (u64)kSortFew && level < 3; ++level) {
    int shift = 0;
    while (((k_hi - k_lo) >> shift) >= (uint32_t)kBins) ++shift;
    cluster_sync();   // every CTA has read the last histogram
    clear_bins(sh);
    if (threadIdx.x == 0) sh.j_lo = sh.j_hi = kBins - 1;
    __syncthreads();
    const float v_lo = logit_of(k_lo), v_hi = logit_below(k_hi);
    part.rare([&](float v) { v = capped(s, v); return v >= v_lo && v <= v_hi; }, [&](float v, int) {
      v = capped(s, v);
      const uint32_t b = (k_hi - key_of(v)) >> shift;
      atomicAdd(&sh.cnt[b], 1u);
      atomicAdd(&sh.lo[b], (uint32_t)(ex2_eighth(fminf((float)bin - eighths(s, v), 0.f)) * 16384.f));   // cut off: within 1
    });
    cluster_sync();
    merge_bins(sh, ctas, true, c, m);
    const u64 ci = block_incl(c[0] + c[1], sh.red, &all), mi = block_incl(m[0] + m[1], sh.red, &all);
    auto low = [&](u64 sum) { return m_lo + (float)bin_mass(sh.eighth, sum << 14, bin) * (1.f - 2e-5f); };
    auto high = [&](u64 sum, u64 n) { return m_hi + (float)bin_mass(sh.eighth, (sum + n) << 14, bin) * (1.f + 2e-5f); };
    find(high(mi - m[1], ci - c[1]) >= want_lo, high(mi, ci) >= want_lo, low(mi - m[1]) >= want_hi, low(mi) >= want_hi);
    const int last = (int)((k_hi - k_lo) >> shift), lo = min(sh.j_lo, last), hi = min(sh.j_hi, last);
    if ((lo & ~1) == b0) sh.c_lo = lo & 1 ? ci - c[1] : ci - c[1] - c[0], sh.m_lo = lo & 1 ? mi - m[1] : mi - m[1] - m[0];
    if ((hi & ~1) == b0) sh.c_hi = hi & 1 ? ci : ci - c[1];
    __syncthreads();
    inside = sh.c_hi - sh.c_lo;
    m_hi = high(sh.m_lo, sh.c_lo), m_lo = low(sh.m_lo);
    const uint32_t to_lo = (uint32_t)(hi + 1) << shift;   // 0: 2^32
    if (k_hi - k_lo >= to_lo && to_lo != 0) k_lo = k_hi - to_lo + 1;
    k_hi -= (uint32_t)lo << shift;
  }
  *k_lo_out = k_lo, *k_hi_out = k_hi;
  return inside <= (u64)kCap;
}

// The row of a cluster when there are more rows than run at once.  Rows cost up to
// seven times one another by what is asked of them, so each 512 go in four classes,
// costly ones first: top-p over the whole row, other samples of a whole row, top-k,
// greedy rows.  192 rows of 262144 with mixed settings, in the order given: an
// SM works 64 % of the time, the rest is the wait for the last rows.
__device__ __forceinline__ int row_in_order(const Params& p, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = (int)blockIdx.y & ~(kThr - 1), r = base + threadIdx.x;
  int cls = 4;
  if (r < p.rows) {
    const float temp = p.temperature ? p.temperature[r] : 1.f, top_p = p.top_p ? p.top_p[r] : 1.f;
    const int k = p.top_k ? p.top_k[r] : 0;
    cls = !(temp > 0.f) || top_p <= 0.f || k == 1 ? 3 : k > 0 && k < p.V ? 2 : top_p < 1.f ? 0 : 1;
  }
  const uint32_t b0 = __ballot_sync(0xffffffffu, cls == 0), b1 = __ballot_sync(0xffffffffu, cls == 1),
                 b2 = __ballot_sync(0xffffffffu, cls == 2);
  if (lane == 0) sh.red32[warp] = __popc(b0) | __popc(b1) << 10 | __popc(b2) << 20;   // 512 rows: 10 bits each
  __syncthreads();
  const uint32_t n = lane < kWarpsS ? sh.red32[lane] : 0u;
  const uint32_t all = __reduce_add_sync(0xffffffffu, n), before = __reduce_add_sync(0xffffffffu, lane < warp ? n : 0u);
  const uint32_t mine = cls == 0 ? b0 : cls == 1 ? b1 : cls == 2 ? b2 : b0 | b1 | b2;
  int at = __popc(mine & ((1u << lane) - 1u));   // of the class before this one
  if (cls < 3) at += before >> 10 * cls & 0x3ffu;
  else at = (int)threadIdx.x - at - (before & 0x3ffu) - (before >> 10 & 0x3ffu) - (before >> 20);
  if (cls > 0) at += all & 0x3ffu;
  if (cls > 1) at += all >> 10 & 0x3ffu;
  if (cls > 2) at += all >> 20;
  if (cls < 4 && base + at == (int)blockIdx.y) sh.row = r;
  __syncthreads();
  return sh.row;
}

template <typename T, bool KEEP>
__global__ void __launch_bounds__(kThr, KEEP ? 1 : 2) sample_kernel(const __grid_constant__ Params p) {
  __shared__ Shared sh;
  uint32_t rank, ctas;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) sh.n_list = 0, sh.first = 0x7fffffff;
  if (threadIdx.x < 8) sh.eighth[threadIdx.x] = kEighth[threadIdx.x];
  clear_bins(sh);
  pdl_wait();
  const int row = p.order ? row_in_order(p, sh) : (int)blockIdx.y;
  const T* z = static_cast<const T*>(p.z) + row * p.stride;
  const bool vec = (reinterpret_cast<uintptr_t>(z) & 15) == 0;
  const int i0 = min((int)rank * p.range, p.V), i1 = min(i0 + p.range, p.V);
  Part<T, KEEP> part;
  part.row = z, part.i0 = i0, part.i1 = i1, part.vec = vec;
  part.load();

  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int k_in = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = fminf(fmaxf(p.u[row], 0.f), 0.99999994f);
  const bool has_k = k_in > 0 && k_in < p.V;
  const bool has_p = top_p < 1.f;
  const bool has_m = min_p > 0.f;

  // ---- A: the maximum (fmaxf passes over a NaN)
  float top = -CUDART_INF_F;
  {
    part.light([&](float v, int) { top = fmaxf(top, v); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.red32[warp] = __float_as_uint(top);
    __syncthreads();
    if (warp == 0) {
      top = lane < kWarpsS ? __uint_as_float(sh.red32[lane]) : -CUDART_INF_F;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) sh.top = top;
    }
    cluster_sync();
    top = lane < (int)ctas ? __uint_as_float(ld_cluster_u32(tc::cluster_addr(&sh.top, lane))) : -CUDART_INF_F;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  const bool nothing = top == -CUDART_INF_F;
  const bool greedy = !(temp > 0.f) || k_in == 1 || top_p <= 0.f;
  if (nothing || greedy) {   // the same in every CTA of the cluster
    if (!nothing) {
      int first = 0x7fffffff;
      part.light([&](float v, int i) { first = v == top ? min(first, i) : first; });
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane == 0 && first != 0x7fffffff) atomicMin(&sh.first, first);
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
      int first = 0x7fffffff;
      for (uint32_t r = 0; r < ctas; ++r) first = min(first, (int)ld_cluster_u32(tc::cluster_addr(&sh.first, r)));
      p.token[row] = nothing ? -1 : first;
      if (p.logprob) p.logprob[row] = nothing ? -CUDART_INF_F : 0.f;
    }
    cluster_sync();   // no CTA leaves while another reads its shared memory
    return;
  }
  const Scale s = make_scale(top, temp, min_p);

  int last = kBins - 1;          // last bin that S can reach
  uint32_t n_cand = 0xffffffffu;   // elements up to it
  u64 total = 0;                 // mass of the row (top-p without top-k)
  u64 cnt[2] = {0, 0}, mant[2] = {0, 0};   // this thread's two bins of the row's histogram
  const bool row_mass = has_p && !has_k;
  // E's first half: the range of keys that holds the border
  uint32_t near_lo = 0, near_hi = 0;
  const bool near = row_mass && narrow(part, sh, s, top_p, p.range, ctas, &near_lo, &near_hi);
  if (row_mass && !near) {
    cluster_sync();   // every CTA has read the last histogram
    clear_bins(sh);
    __syncthreads();
  }
  if (!near && (has_k || has_p || has_m)) {
    // ---- B: histogram over the row, with masses for top-p without top-k
    // (which goes by the mass of the whole row)
    if (row_mass) {
      part.heavy([&](float v, int) {
        v = capped(s, v);
        const float q = eighths(s, v);
        if (q < (float)kBins) {
          float nf;
          const int n = whole(q, &nf);
          add_to_bin(sh, n, mantissa(s, v, q, nf));
        }
      });
    } else {
      part.light([&](float v, int) {
        const float q = eighths(s, capped(s, v));
        if (q < (float)kBins) atomicAdd(&sh.cnt[(int)q], 1u);
      });
    }
    cluster_sync();
    merge_bins(sh, ctas, row_mass, cnt, mant);
    if (row_mass)
      block_incl(bin_mass(sh.eighth, mant[0], 2 * threadIdx.x) + bin_mass(sh.eighth, mant[1], 2 * threadIdx.x + 1), sh.red, &total);
    u64 all;
    const u64 incl = block_incl(cnt[0] + cnt[1], sh.red, &all);
    const u64 c0 = incl - cnt[1], c1 = incl;   // elements up to bin 2 tid and 2 tid + 1
    // a lower bound on the mass up to a bin: 2^-((n + 1)/8) per element
    const int b0 = 2 * threadIdx.x;
    const float h0 = exp2f(-0.125f * b0), q = 0.91700404f;   // 2^(-1/8)
    float mtot;
    const float mass = block_incl(((float)cnt[0] + (float)cnt[1] * q) * h0 * q * 0.9999f, reinterpret_cast<float*>(sh.red32), &mtot);
    const float m0 = mass - (float)cnt[1] * q * q * h0;   // up to bin b0 (a little less)
    // The first bin where one of the sets must have ended.  With both top-k and
    // top-p the mass of all of S_k is wanted, so only top-k ends it.
    const float target = has_p ? top_p * ((float)total * 2.2737368e-13f) * 1.0002f : CUDART_INF_F;
    const float mbin = has_m ? -8.f * log2f(fminf(min_p, 1.f)) + 1.f : 2000.f;
    const bool k_only = has_k && has_p;
    const bool e0 = (has_k && c0 >= (u64)k_in) || c0 == all || (!k_only && (m0 >= target || (float)b0 >= mbin));
    const bool e1 = (has_k && c1 >= (u64)k_in) || c1 == all || (!k_only && (mass >= target || (float)(b0 + 1) >= mbin));
    int mine = e0 ? b0 : e1 ? b0 + 1 : kBins - 1;
    mine = __reduce_min_sync(0xffffffffu, mine);
    __syncthreads();
    if (lane == 0) sh.red32[warp] = (uint32_t)mine;
    __syncthreads();
    for (int w = 0; w < kWarpsS; ++w) last = min(last, (int)sh.red32[w]);
    if (b0 == (last & ~1)) sh.scan_total = (last & 1) ? c1 : c0;
    __syncthreads();
    n_cand = (uint32_t)sh.scan_total;
  }

  if (n_cand <= (uint32_t)kCap) {
    // ---- C: the candidates into the leader
    const uint32_t list0 = tc::cluster_addr(sh.list, 0), count0 = tc::cluster_addr(&sh.n_list, 0);
    const float lim = (float)(last + 1);
    part.rare([&](float v) { return eighths(s, capped(s, v)) < lim; }, [&](float v, int i) {
      uint32_t at;
      asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(at) : "r"(count0) : "memory");
      const u64 c = ((u64)~key_of(capped(s, v)) << 32) | (uint32_t)i;
      if (at < (uint32_t)kCap) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(list0 + 8 * at), "l"(c) : "memory");
    });
    cluster_sync();
    if (rank != 0) return;   // only the leader's own memory is used from here
    const int n = (int)min(n_cand, (uint32_t)kCap);
    if (n <= kCount) {
      // each element's place: how many come before it (two threads count)
      const u64 c = (int)(threadIdx.x >> 1) < n ? sh.list[threadIdx.x >> 1] : ~0ull;
      int place = 0;
      for (int j = threadIdx.x & 1; j < n; j += 2) place += sh.list[j] < c;
      place += __shfl_xor_sync(0xffffffffu, place, 1);
      __syncthreads();
      if ((threadIdx.x & 1) == 0 && (int)(threadIdx.x >> 1) < n) sh.list[place] = c;
      __syncthreads();
    } else {
      int n2 = 2 * kCount;
      while (n2 < n) n2 <<= 1;
      for (int i = n + threadIdx.x; i < n2; i += kThr) sh.list[i] = ~0ull;
      bitonic(sh.list, n2);
    }
    // cut: thread i holds the kPer elements from kPer i on
    constexpr int kPer = kCap / kThr;
    u64 w[kPer], mass_k = 0, sum = 0;
    const int nk = has_k ? min(n, k_in) : n;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = kPer * threadIdx.x + j;
      w[j] = i < nk ? weight(sh.eighth, s, logit_of(~(uint32_t)(sh.list[i] >> 32))) : 0ull;
      sum += w[j];
    }
    const u64 incl = block_incl(sum, sh.red, &mass_k);
    // kept while the mass before it is below this
    const u64 limit = has_p ? times(has_k ? mass_k : total, top_p, true) : ~0ull;
    u64 before = incl - sum, kept = 0;
    int keep = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = kPer * threadIdx.x + j;
      const bool k = i < nk && (i == 0 || (before < limit && (!has_m || passes_minp(sh.eighth, s, logit_of(~(uint32_t)(sh.list[i] >> 32))))));
      before += w[j];
      keep += k;
      kept += k ? w[j] : 0ull;
    }
    u64 mass;
    block_incl(kept, sh.red, &mass);
    keep = (int)__reduce_add_sync(0xffffffffu, (unsigned)keep);
    __syncthreads();
    if (lane == 0) sh.red32[warp] = (uint32_t)keep;
    // the first weights, beside the elements
    u64* wt = reinterpret_cast<u64*>(sh.cnt);
    static_assert(sizeof(sh.cnt) >= kCount * 8, "the weights take the place of the bins");
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (kPer * threadIdx.x + j < kCount) wt[kPer * threadIdx.x + j] = w[j];
    __syncthreads();
    keep = 0;
    for (int x = 0; x < kWarpsS; ++x) keep += (int)sh.red32[x];
    // the first running mass, in vocabulary order, above the goal
    const u64 goal = min(times(mass, u, false), mass - 1);
    auto pick = [&](int index, uint32_t inverted_key) {
      p.token[row] = index;
      if (p.logprob) p.logprob[row] = log_prob(p, row, s.top, logit_of(~inverted_key), mass);
    };
    if (u == 0.f) {   // the first of S, whose weight may be less than a unit
      int first = 0x7fffffff;
      for (int i = threadIdx.x; i < keep; i += kThr) first = min(first, (int)(uint32_t)sh.list[i]);
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane == 0) atomicMin(&sh.first, first);
      __syncthreads();
      for (int i = threadIdx.x; i < keep; i += kThr)
        if ((int)(uint32_t)sh.list[i] == sh.first) pick(sh.first, (uint32_t)(sh.list[i] >> 32));
    } else if (keep <= kCount) {
      const int i = threadIdx.x >> 1;
      const uint32_t at = i < keep ? (uint32_t)sh.list[i] : 0u;
      u64 run = 0;
      for (int j = threadIdx.x & 1; j < keep; j += 2) run += (uint32_t)sh.list[j] < at ? wt[j] : 0ull;
      run += __shfl_xor_sync(0xffffffffu, run, 1);
      if ((threadIdx.x & 1) == 0 && i < keep && run <= goal && run + wt[i] > goal) pick((int)at, (uint32_t)(sh.list[i] >> 32));
    } else {
      int n2 = 2 * kCount;
      while (n2 < keep) n2 <<= 1;
      for (int i = threadIdx.x; i < n2; i += kThr) {
        const u64 c = sh.list[i];
        sh.list[i] = i < keep ? (c << 32) | (c >> 32) : ~0ull;
      }
      bitonic(sh.list, n2);
      sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        w[j] = i < keep ? weight(sh.eighth, s, logit_of(~(uint32_t)sh.list[i])) : 0ull;
        sum += w[j];
      }
      u64 run = block_incl(sum, sh.red, &mass) - sum;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        if (i < keep && run <= goal && run + w[j] > goal) pick((int)(sh.list[i] >> 32), (uint32_t)sh.list[i]);
        run += w[j];
      }
    }
    return;
  }

  // ---- D: the threshold by refinement.  Kept: key > thr_key, and the first
  // thr_ties (by index) of those equal to it.
  uint32_t thr_key = 0;
  u64 thr_ties = ~0ull;
  if (!near && (has_k || has_p)) {
    if (has_p && has_k) {   // the masses too, up to the last bin that matters
      cluster_sync();       // every CTA has read the counts
      clear_bins(sh);
      __syncthreads();
      const float lim = (float)(last + 1);
      part.rare([&](float v) { return eighths(s, capped(s, v)) < lim; }, [&](float v, int) {
        v = capped(s, v);
        const float q = eighths(s, v);
        float nf;
        const int n = whole(q, &nf);
        add_to_bin(sh, n, mantissa(s, v, q, nf));
      });
      cluster_sync();
      merge_bins(sh, ctas, true, cnt, mant);
    }
    u64 mass[2] = {bin_mass(sh.eighth, mant[0], 2 * threadIdx.x), bin_mass(sh.eighth, mant[1], 2 * threadIdx.x + 1)};
    u64 dummy;
    const u64 cnt_incl = block_incl(cnt[0] + cnt[1], sh.red, &dummy);
    const u64 mass_incl = block_incl(mass[0] + mass[1], sh.red, &dummy);

    // Descends into one bin until a single key is left.  by_mass: the first
    // element whose mass including it reaches `goal`; else the goal-th element.
    auto descend = [&](bool by_mass, u64 goal, u64* mass_out) {
      // the crossing bin of the first level
      __syncthreads();
      if (threadIdx.x == 0) sh.cross_bin = -1;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u64 c_in = j ? cnt_incl : cnt_incl - cnt[1], m_in = j ? mass_incl : mass_incl - mass[1];
        const u64 c_ex = c_in - cnt[j], m_ex = m_in - mass[j];
        const bool hit = by_mass ? m_ex < goal && m_in >= goal : c_ex < goal && c_in >= goal;
        if (hit) sh.cross_bin = 2 * threadIdx.x + j, sh.cross_cnt = (uint32_t)c_ex, sh.cross_mass = m_ex;
      }
      __syncthreads();
      const int bin = sh.cross_bin;
      if (bin < 0) {   // the goal lies behind everything that counts
        thr_key = 0, thr_ties = ~0ull;
        *mass_out = dummy;
        return;
      }
      u64 c_before = sh.cross_cnt, m_before = sh.cross_mass;
      // the keys of the bin: eighths() is monotone in the logit, so they are a range
      uint32_t k_lo, k_hi;   // keys of the bin: [k_lo, k_hi]
      {
        k_lo = first_key(s, (float)(bin + 1));
        k_hi = bin == 0 ? key_of(s.top) : first_key(s, (float)bin) - 1;
      }
      for (;;) {
        const uint32_t width = k_hi - k_lo;   // keys - 1
        int shift = 0;
        while ((width >> shift) >= (uint32_t)kBins) ++shift;
        cluster_sync();   // every CTA has read the last histogram
        clear_bins(sh);
        __syncthreads();
        // (on the logits: the key of a NaN lies outside)
        const float v_lo = logit_of(k_lo), v_hi = logit_below(k_hi);
        part.rare([&](float v) { v = capped(s, v); return v >= v_lo && v <= v_hi; }, [&](float v, int) {
          v = capped(s, v);
          const int b = (int)((k_hi - key_of(v)) >> shift);
          if (has_p) add_to_bin(sh, b, mantissa(s, v, eighths(s, v), (float)bin));
          else atomicAdd(&sh.cnt[b], 1u);
        });
        cluster_sync();
        u64 c[2], m[2];
        merge_bins(sh, ctas, has_p, c, m);
        u64 t;
        const u64 ci = block_incl(c[0] + c[1], sh.red, &t);
        const u64 m_sub[2] = {bin_mass(sh.eighth, m[0], bin), bin_mass(sh.eighth, m[1], bin)};
        const u64 mi = block_incl(m_sub[0] + m_sub[1], sh.red, &t);
        if (threadIdx.x == 0) sh.cross_bin = -1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u64 c_in = c_before + (j ? ci : ci - c[1]), m_in = m_before + (j ? mi : mi - m_sub[1]);
          const u64 c_ex = c_in - c[j], m_ex = m_in - m_sub[j];
          const bool hit = by_mass ? m_ex < goal && m_in >= goal : c_ex < goal && c_in >= goal;
          if (hit) sh.cross_bin = 2 * threadIdx.x + j, sh.cross_cnt = (uint32_t)c_ex, sh.cross_mass = m_ex;
        }
        __syncthreads();
        int sub = sh.cross_bin;
        if (sub < 0) {   // rounding of the bin masses: the goal is the bin's very end
          // the last occupied sub-bin
          __syncthreads();
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (c[j]) atomicMax(&sh.cross_bin, 2 * (int)threadIdx.x + j);
          __syncthreads();
          sub = sh.cross_bin;
          if (2 * (int)threadIdx.x == (sub & ~1)) {
            const int j = sub & 1;
            sh.cross_cnt = (uint32_t)(c_before + (j ? ci : ci - c[1]) - c[j]);
            sh.cross_mass = m_before + (j ? mi : mi - m_sub[1]) - m_sub[j];
          }
          __syncthreads();
        }
        c_before = sh.cross_cnt, m_before = sh.cross_mass;
        const uint32_t hi = k_hi - ((uint32_t)sub << shift);
        const uint32_t span = (1u << shift) - 1u;
        k_lo = hi - k_lo > span ? hi - span : k_lo;
        k_hi = hi;
        if (shift == 0) {
          thr_key = k_hi;
          const float v = logit_of(k_hi);
          const u64 w = weight_of(sh.eighth, mantissa(s, v, eighths(s, v), (float)bin), bin);
          const u64 rest = goal > (by_mass ? m_before : c_before) ? goal - (by_mass ? m_before : c_before) : 1ull;
          thr_ties = by_mass ? (w ? (rest + w - 1) / w : ~0ull) : rest;
          *mass_out = m_before + w * (by_mass ? 0ull : thr_ties);
          return;
        }
      }
    };
    u64 mass_k = dummy;
    if (has_k) descend(false, (u64)k_in, &mass_k);
    if (has_p) {
      const uint32_t kk = thr_key;
      const u64 kt = thr_ties;
      u64 unused;
      descend(true, max(times(has_k ? mass_k : total, top_p, true), 1ull), &unused);
      if (has_k && (thr_key < kk || (thr_key == kk && thr_ties > kt))) thr_key = kk, thr_ties = kt;
    }
  }

  // masses and ties of the segments of this CTA's range
  cluster_sync();   // sh.list / sh.seg are free, every histogram read
  const int n_seg = (i1 - i0 + kSeg - 1) / kSeg;
  const bool cuts = thr_key != 0;
  u64* const seg = near ? reinterpret_cast<u64*>(sh.cnt) : sh.seg;   // (the list is in use beside it)
  static_assert(sizeof(sh.cnt) + sizeof(sh.lo) == sizeof(sh.seg) && offsetof(Shared, lo) == sizeof(sh.cnt), "two rows of bins");
  const float cut = cuts ? logit_of(thr_key) : -CUDART_INF_F;   // (copies: descend() holds references to the others)
  const u64 cut_ties = thr_ties;
  auto kept = [&](float v) { return v > cut && (!has_m || passes_minp(sh.eighth, s, v)); };
  auto tied = [&](float v) { return cuts && v == cut && (!has_m || passes_minp(sh.eighth, s, v)); };
  // four consecutive indices of a segment per lane
  auto load4 = [&](int g, float (&v)[4]) {
    load_logits<T, 4>(z, i0 + g * kSeg + 4 * lane, i1, vec, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = capped(s, v[k]);
  };
  // the sum of the lanes' masses, each below 2^45: two pieces of 23 bits
  auto lanes_sum = [](u64 v) {
    const u64 lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7fffffu);
    return lo + ((u64)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 23)) << 23);
  };
  // near: kept is what lies above the range that holds the border, and the first of the range
  const float v_min = near && has_m ? logit_of(minp_key(sh.eighth, s)) : -CUDART_INF_F, v_hi = logit_below(near_hi);
  auto above_range = [&](float v) { return v > v_hi && v >= v_min; };
  u64 last_kept = 0;
  if (near) {
    // ---- E: the mass of the row, those above the range, and its elements to the leader
    const float v_lo = fmaxf(logit_of(near_lo), v_min);
    const uint32_t list0 = tc::cluster_addr(sh.list, 0), count0 = tc::cluster_addr(&sh.n_list, 0);
    u64 row_part = 0;
    float next[4];
    load4(warp, next);
#pragma unroll 1
    for (int g = warp; g < n_seg; g += kWarpsS) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = next[k];
      load4(g + kWarpsS, next);
      u64 sum = 0;
      bool any = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u64 wk = weight(sh.eighth, s, v[k]);
        row_part += wk;
        sum += above_range(v[k]) ? wk : 0ull;
        any |= v[k] <= v_hi && v[k] >= v_lo;
      }
      if (any) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const float x = k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3];
          if (!(x <= v_hi && x >= v_lo)) continue;
          uint32_t at;
          asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(at) : "r"(count0) : "memory");
          const u64 c = ((u64)~key_of(x) << 32) | (uint32_t)(i0 + g * kSeg + 4 * lane + k);
          if (at < (uint32_t)kCap) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(list0 + 8 * at), "l"(c) : "memory");
        }
      }
      __syncwarp();
      sum = lanes_sum(sum);
      if (lane == 0) seg[g] = sum;
    }
    __syncthreads();
    u64 above = 0, cta_row, cta_above;
    for (int g = threadIdx.x; g < n_seg; g += kThr) above += seg[g];
    block_incl(row_part, sh.red, &cta_row);
    block_incl(above, sh.red, &cta_above);
    if (threadIdx.x == 0) sh.mine = cta_row, sh.ties = cta_above;
    cluster_sync();
    u64 unused;
    const u64 row = cluster_sum(&sh.mine, rank, ctas, &unused);
    above = cluster_sum(&sh.ties, rank, ctas, &unused);
    if (rank == 0) {
      const int n = (int)min(sh.n_list, (uint32_t)kCap);
      int n2 = 64;
      while (n2 < n) n2 <<= 1;
      for (int i = n + threadIdx.x; i < n2; i += kThr) sh.list[i] = ~0ull;
      bitonic(sh.list, n2);
      constexpr int kPer = kCap / kThr;
      u64 w[kPer], sum = 0, t;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        w[j] = i < n ? weight(sh.eighth, s, logit_of(~(uint32_t)(sh.list[i] >> 32))) : 0ull;
        sum += w[j];
      }
      u64 before = above + block_incl(sum, sh.red, &t) - sum;
      const u64 limit = max(times(row, top_p, true), 1ull);
      int keep = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        keep += kPer * (int)threadIdx.x + j < n && before < limit;
        before += w[j];
      }
      keep = (int)__reduce_add_sync(0xffffffffu, (unsigned)keep);
      if (threadIdx.x == 0) sh.n_kept = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(&sh.n_kept, keep);
      __syncthreads();
      if (threadIdx.x == 0) sh.last_kept = sh.n_kept ? sh.list[sh.n_kept - 1] : 0ull;
    }
    cluster_sync();
    const int n_kept = (int)ld_cluster_u32(tc::cluster_addr(&sh.n_kept, 0));
    last_kept = ld_cluster_u64(tc::cluster_addr(&sh.last_kept, 0));
    for (int i = threadIdx.x; i < n_kept; i += kThr) {
      const u64 c = ld_cluster_u64(tc::cluster_addr(&sh.list[i], 0));
      const int at = (int)(uint32_t)c - i0;
      if (at >= 0 && at < i1 - i0) atomicAdd(&seg[at / kSeg], weight(sh.eighth, s, logit_of(~(uint32_t)(c >> 32))));
    }
  } else {
    float next[4];
    load4(warp, next);
#pragma unroll 1
    for (int g = warp; g < n_seg; g += kWarpsS) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = next[k];
      load4(g + kWarpsS, next);
      u64 sum = 0;
      uint32_t ties = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u64 wk = weight(sh.eighth, s, v[k]);
        sum += kept(v[k]) ? wk : 0ull;
        ties += tied(v[k]);
      }
      sum = lanes_sum(sum);
      ties = __reduce_add_sync(0xffffffffu, ties);
      if (lane == 0) seg[g] = sum, sh.tie[g] = ties;
    }
  }
  __syncthreads();
  // prefix of the ties: how many of a segment's are kept
  constexpr int kPerS = kMaxSegs / kThr;
  u64 t_sum = 0, m_sum = 0;
  u64 cta_ties, cta_mass, t_run = 0;
  if (cuts) {   // else nothing is tied
    for (int j = 0; j < kPerS; ++j) {
      const int g = threadIdx.x * kPerS + j;
      if (g < n_seg) t_sum += sh.tie[g];
    }
    t_run = block_incl(t_sum, sh.red, &cta_ties) - t_sum;
    if (threadIdx.x == 0) sh.ties = cta_ties;
    cluster_sync();
    u64 before;
    cluster_sum(&sh.ties, rank, ctas, &before);
    t_run += before;
  }
  const u64 w_tie = cuts ? weight(sh.eighth, s, cut) : 0ull;
  const u64 t_first = t_run;
  m_sum = 0;
  for (int j = 0; j < kPerS; ++j) {
    const int g = threadIdx.x * kPerS + j;
    if (g < n_seg) {
      if (cuts) {
        const u64 left = cut_ties > t_run ? cut_ties - t_run : 0ull;
        t_run += sh.tie[g];
        seg[g] += w_tie * min((u64)sh.tie[g], left);
      }
      m_sum += seg[g];
    }
  }
  u64 m_run = block_incl(m_sum, sh.red, &cta_mass) - m_sum;
  if (threadIdx.x == 0) sh.mine = cta_mass;
  cluster_sync();
  u64 before;
  const u64 mass = cluster_sum(&sh.mine, rank, ctas, &before);
  if (u == 0.f) {   // the first of S, whose weight may be less than a unit (the same in every CTA)
    int first = 0x7fffffff;
    part.heavy([&](float x, int i) {
      const float v = capped(s, x);
      const u64 c = (u64)~key_of(v) << 32 | (uint32_t)i;
      const bool in = near ? above_range(v) || (v <= v_hi && c <= last_kept) : kept(v) || tied(v);   // the first that ties is kept
      if (in && eighths(s, v) < (float)kBins) first = min(first, i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&sh.first, first);
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
      first = 0x7fffffff;
      for (uint32_t r = 0; r < ctas; ++r) first = min(first, (int)ld_cluster_u32(tc::cluster_addr(&sh.first, r)));
      p.token[row] = first;
      if (p.logprob) p.logprob[row] = log_prob(p, row, s.top, capped(s, as_float(z[first])), mass);
    }
    cluster_sync();   // no CTA leaves while another reads its shared memory
    return;
  }
  const u64 goal = min(times(mass, u, false), mass - 1);
  m_run += before;
  t_run = t_first;
  if (threadIdx.x == 0) sh.cross_bin = -1;
  __syncthreads();
  for (int j = 0; j < kPerS; ++j) {
    const int g = threadIdx.x * kPerS + j;
    if (g < n_seg) {
      if (m_run <= goal && m_run + seg[g] > goal) {
        sh.cross_bin = g;
        sh.cross_mass = m_run;
        sh.scan_total = t_run;
      }
      m_run += seg[g];
      t_run += cuts ? sh.tie[g] : 0u;
    }
  }
  __syncthreads();
  if (warp == 0 && sh.cross_bin >= 0) {
    const int i = i0 + sh.cross_bin * kSeg + 4 * lane;
    float v[4];
    load4(sh.cross_bin, v);
    u64 w[4], sum = 0;
    uint32_t ties = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) ties += tied(v[k]);
    u64 t_at = sh.scan_total + warp_incl(ties) - ties;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u64 c = (u64)~key_of(v[k]) << 32 | (uint32_t)(i + k);
      const bool in = near ? above_range(v[k]) || (v[k] <= v_hi && c <= last_kept) : kept(v[k]);
      w[k] = in ? weight(sh.eighth, s, v[k]) : 0ull;
      if (tied(v[k])) w[k] = t_at++ < cut_ties ? w_tie : 0ull;
      sum += w[k];
    }
    u64 run = sh.cross_mass + warp_incl(sum) - sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (run <= goal && run + w[k] > goal) {
        p.token[row] = i + k;
        if (p.logprob) p.logprob[row] = log_prob(p, row, s.top, v[k], mass);
      }
      run += w[k];
    }
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

template <typename T, bool KEEP>
static int launch_k(const Params& p, int rows, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, rows);
  cfg.blockDim = dim3(kThr);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<T, KEEP>, p);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "sampling launch");
}

template <typename T>
static int launch(const Params& p, int rows, int cluster, bool keep, cudaStream_t s) {
  return keep ? launch_k<T, true>(p, rows, cluster, s) : launch_k<T, false>(p, rows, cluster, s);
}

}  // namespace sample

int launch_logits_sample(const void* z, long long stride, int dtype, int rows, int V, const float* u,
                         const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                         int32_t* token, float* logprob, const DeviceInfo& dev, cudaStream_t s) {
  sample::Params p = {z, stride, u, temperature, top_k, top_p, min_p, token, logprob, V, 0, rows, 0};
  // CTAs per row.  Few rows: eight, one CTA per SM with its part of the row in
  // registers (a cluster lies in one GPC, so not every SM can be used; 8 rows of
  // 262144: 15.9 us for top-64, against 22 with four that read again).  Up to as
  // many rows as run at once with eight, two CTAs per SM that read the row again
  // from L2: eight, as a row's time counts where settings differ (32 rows: 52 us
  // for mixed settings against 69 with four, top-64 for all 24.6 against 25.0,
  // top-p 0.9 for all 73 against 68).  More: four, as every phase that one CTA runs
  // alone idles fewer (64 rows: top-64 32 us against 45, top-p 100 against 139; 192
  // rows, mixed: 151 against 184).  Not more indices per CTA than a 32-bit bin
  // holds, nor CTAs for a few thousand indices.
  const bool few = rows * 8 <= dev.sms * 2 / 3;
  int cluster = rows * 8 <= dev.sms * 7 / 4 ? 8 : 4;   // 7/8 of the places of two CTAs per SM
  while (cluster > 1 && V <= 2048 * cluster) cluster >>= 1;
  while (V > cluster * sample::kSeg * sample::kMaxSegs) cluster <<= 1;
  const int segs = (V + sample::kSeg * cluster - 1) / (sample::kSeg * cluster);
  p.range = segs * sample::kSeg;
  p.order = rows * cluster > 2 * dev.sms && (temperature || top_k || top_p);
  const bool keep = few && p.range <= sample::kKeep * sample::kThr;
  return dtype == Q4_F32   ? sample::launch<float>(p, rows, cluster, keep, s)
         : dtype == Q4_F16 ? sample::launch<__half>(p, rows, cluster, keep, s)
                           : sample::launch<__nv_bfloat16>(p, rows, cluster, keep, s);
}

}  // namespace q4w
