// Verification of drafted tokens: which of a user's k drafts stand, and the token
// behind the last of them, from given random numbers.
//
// With p_j = softmax(z_j / T) of the target's rows and q_j = softmax(y_j / T) of the
// draft model's (all on x_j where there are none): draft j stands if u_j q_j(x_j) <
// p_j(x_j); with n the drafts before the first that falls, the next token is drawn by
// u_k from max(p_n - q_n, 0) where draft n fell, from p_n where there was none left.
//
// Kernels, each behind the one before it:
//   rows    the maximum and the sum of weights (greedy users: the maximum's lowest index) of a
//           part of a row per CTA, 64 bytes a thread at once and as many on their way.  HBM
//           bounds it.  Rows that no outcome can need are not read: those behind a place
//           without a draft, and the draft model's of greedy users.
//   choose  a CTA per user joins the parts, finds n and lists the rows whose exact masses are
//           wanted: row n of the target, and of the draft model where a draft fell.  (Few users:
//           every CTA of the next kernel does it for itself.)
//   sums    exact masses of 256-index segments of the listed rows.  The segments of all
//           of them form one line that is cut into equal shares: users need none, one or two
//           rows, and a grid over users left SMs idle half of the time.  The CTA that finishes a
//           row last draws the token where it comes from p_n alone (or from p_n without x_n:
//           drafts without probabilities).
//   rest    segments' masses of max(p_n - q_n, 0), shared out alike; the last CTA draws from them.
// Exact weights are integers (q4w_weights.cuh) of some 30 instructions an element, of which the
// listed rows take one in five; the first kernel's sums are plain fp32 (a dozen instructions
// with the maximum, and an ex2.approx).  They decide whether a draft stands and give its log
// probability, but no border between two tokens is drawn by them.  They are good to 2^-16:
// 2^-22 of ex2.approx for an element and for each of up to 34 changes of the reference, the
// argument's two roundings (2^-23 ln 2 times up to 20, as a million weights cannot have their mass
// deeper), and some 53 additions of 2^-24; errors of random signs leave about 2^-23.
// The rest's probabilities are integers too: the mantissas times 2^(-j/8) / mass, 32 bits formed
// once per row, so that p - q of an element costs two weights and a subtraction.  They are good to 2^-28
// of themselves, as the weights are: the law of a token, over drafts drawn from q, to 2^-27.
//
// Measured (f32, V = 262144): 64 users with up to four drafts, 0 to 4 there (336 MB read of
// 604): rows 50 us (6.5 TB/s), sums 36, rest 23, from a graph 110.  One user of four drafts 18.4
// from a graph: latency of three kernels and, at the end of each draw, of a count, a scan, a
// segment and a logarithm in fp64 (formed beside the search).
#include <math_constants.h>

#include "q4w_device.cuh"
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"
#include "q4w_weights.cuh"

namespace q4w {
namespace verify {

using sample::as_float;
using sample::capped;
using sample::eighths;
using sample::make_scale;
using sample::mantissa;
using sample::mantissas;
using sample::Pair;
using sample::Scale;
using sample::shift_right;
using sample::times;
using sample::u64;
using sample::weight;
using sample::whole;

constexpr int kThr = 256;
constexpr int kWarpsV = kThr / 32;
constexpr int kMaxBatches = 16;         // of a CTA of the first kernel
constexpr int kSeg = 256;               // indices of a segment: eight neighbours per lane
constexpr int kMaxChunks = 128;         // CTAs per row of the first kernel
constexpr int kRowCtas = 12;            // of the first kernel, per SM, that make further batches a CTA worth while
constexpr int kResident = 3;            // CTAs per SM of the exact passes (two or four: 1 % slower)
constexpr int kMaxDrafts = 64;
constexpr int kFewUsers = 2;            // FEW of sums_kernel: each user more is 2 us, the kernel that it saves 3 to 5
constexpr int kUnit = 53;               // the rest's masses are in units of 2^-53

// What follows the drafts that stand.
enum { kNothing, kLargest, kTarget, kRest };
// A row whose exact masses are wanted, or a user whose next token comes from the rest.
struct __align__(16) Unit {
  int user, n, kind;
  int without;          // the index that is left out of p_n, or -1
  float t, top, top_q;  // top: of the row; of the rest's users both rows'
  int drafted;          // the row is the draft model's
};

struct Params {
  const void *z, *y;              // [b][k + 1][V], [b][k][V] or NULL
  long long z_user, z_row, y_user, y_row;
  const int32_t* x;               // [b][k]
  const float* u;                 // [b][k + 1]
  const float* temperature;       // [b], NULL: 1
  int32_t *tokens, *accepted;     // [b][k + 1], [b]
  float* logprobs;                // [b][k + 1] or NULL
  int b, k, V, chunks, batches;      // of a row: CTAs, each of so many batches
  int n_segs, ctas;               // segments of a row; CTAs of the other kernels
  float2* rows;                   // [b][2 k + 1][chunks]: maximum and sum (or index)
  float2* joined;                 // [b][k + 1]: of the target's rows
  int* units;                     // how many there are of the two lists
  Unit *list, *rest;              // [2 b], [b]
  u64* mass;                      // [b][2]: of p_n's and q_n's row, where a rest is wanted
  u64* seg;                       // [b][2][n_segs]: masses of p_n's row's segments, of the rest's
  unsigned* done;                 // [b][2]: CTAs that have finished with a user
};

// A weight relative to `top` by ex2.approx, for rows whose sums need no more.
struct Cheap {
  float ch, cl, least;   // log2(e) / T in two pieces; differences below `least` weigh nothing
};
__device__ __forceinline__ float temperature_of(const Params& p, int user) {
  const float t = p.temperature ? p.temperature[user] : 1.f;
  return t > 0.f ? fminf(fmaxf(t, 1e-36f), 1.2676506e30f) : 0.f;   // 0: greedy; 2^100 at most, so that -inf / T is -inf
}
__device__ __forceinline__ Cheap make_cheap(float t) {
  const Scale s = make_scale(0.f, t, 0.f);
  return {s.ch * 0.125f, s.cl * 0.125f, -16000.f / s.ch};
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (fmaxf passes over a NaN: it weighs nothing)
__device__ __forceinline__ float cheap_weight(const Cheap& c, float v, float top) {
  const float d = fmaxf(v - top, c.least);
  return ex2(fmaf(d, c.ch, d * c.cl));
}

// Drafts of a user before the first that is none.  Whole warps.
__device__ __forceinline__ int drafts_of(const Params& p, int user) {
  const int lane = threadIdx.x & 31;
  const int32_t* x = p.x + (long long)user * p.k;
  for (int j = 0; j < p.k; j += 32) {
    const int v = j + lane < p.k ? x[j + lane] : -1;
    const uint32_t none = __ballot_sync(0xffffffffu, v < 0 || v >= p.V);
    if (none) return j + __ffs(none) - 1;
  }
  return p.k;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Params& p, int user, int row) {
  return row <= p.k ? static_cast<const T*>(p.z) + user * p.z_user + row * p.z_row
                    : static_cast<const T*>(p.y) + user * p.y_user + (row - p.k - 1) * p.y_row;
}
// Rows 0 .. k are the target's, the others the draft model's.
__device__ __forceinline__ bool needed(const Params& p, int row, int held, bool greedy) {
  return row <= p.k ? row <= held : !greedy && row - p.k - 1 < held;
}

// What a thread loads in one go: 64 bytes, in 16-byte pieces that a CTA's threads take in turn.
template <typename T>
struct Batch {
  static constexpr int E = 16 / sizeof(T), N = 4;
  uint4 v[N];
  __device__ __forceinline__ void load(const T* z, int i, int V) {
#pragma unroll
    for (int a = 0; a < N; ++a, i += E * kThr) {
      if (i + E <= V) {
        v[a] = *reinterpret_cast<const uint4*>(z + i);
      } else {
        v[a] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);   // NaN
        T* e = reinterpret_cast<T*>(&v[a]);
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (i + j < V) e[j] = z[i + j];
      }
    }
  }
  __device__ __forceinline__ float at(int j) const { return as_float(reinterpret_cast<const T*>(v)[j]); }
};

// A thread's running maximum (starting at -inf) and the sum of weights relative to it.
struct Running {
  float top, sum;
  __device__ __forceinline__ void add(const Cheap& c, float (&v)[16]) {
    float m = fmaxf(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < 16; j += 2) asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v[j]), "f"(v[j + 1]));
    if (m > top) {
      if (m == CUDART_INF_F) {   // counts as the largest number
        m = CUDART_MAX_NORMAL_F;
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = v[j] == CUDART_INF_F ? m : v[j];
      }
      if (m > top) sum *= cheap_weight(c, top, m), top = m;
    }
    // cheap_weight() of two at once
    const f2_t below = f2_pack(-top, -top), ch = f2_pack(c.ch, c.ch), cl = f2_pack(c.cl, c.cl);
    f2_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float d0, d1;
      f2_unpack(f2_add(f2_pack(v[2 * j], v[2 * j + 1]), below), d0, d1);
      const f2_t d = f2_pack(fmaxf(d0, c.least), fmaxf(d1, c.least));
      f2_unpack(f2_fma(d, ch, f2_mul(d, cl)), d0, d1);
      w[j] = f2_pack(ex2(d0), ex2(d1));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < o; ++j) w[j] = f2_add(w[j], w[j + o]);
    float even, odd;
    f2_unpack(w[0], even, odd);
    sum += even + odd;
  }
};

// (Five CTAs an SM, 48 registers, with 20 bytes of spills for 16-bit logits: 16 users of 100003 bf16 logits in
// nine rows 27.2 us in all; four 28.2; six, which spill more, 29.4.)
template <typename T>
__global__ void __launch_bounds__(kThr, 5) rows_kernel(const __grid_constant__ Params p) {
  __shared__ float2 red[kWarpsV];
  const int chunk = blockIdx.x, row = blockIdx.y, user = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (chunk == 0 && row == 0 && threadIdx.x < 2) {
    p.done[2 * user + threadIdx.x] = 0, p.mass[2 * user + threadIdx.x] = 0;
    if (user == 0) p.units[threadIdx.x] = 0;
  }
  const float t = temperature_of(p, user);
  const bool greedy = t == 0.f;
  if (row > 0 && !needed(p, row, drafts_of(p, user), greedy)) return;

  // The row's first elements up to a 16-byte boundary go to the first chunk.
  constexpr int E = Batch<T>::E, kPer = Batch<T>::N * E, kStep = kPer * kThr;
  const T* z = row_of<T>(p, user, row);
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / (int)sizeof(T), p.V);
  int i = head + chunk * p.batches * kStep + E * (int)threadIdx.x;
  Batch<T> now, next;
  next.load(z, i, p.V);
  float extra = CUDART_NAN_F;
  if (chunk == 0 && threadIdx.x < head) extra = as_float(z[threadIdx.x]);

  float2* out = p.rows + ((long long)user * (2 * p.k + 1) + row) * p.chunks + chunk;
  if (greedy) {
    float top = -CUDART_INF_F;
    int first = 0x7fffffff;
    if (extra > top) top = extra, first = threadIdx.x;
    for (int n = 0; n < p.batches; ++n) {
      now = next;
      if (n + 1 < p.batches) next.load(z, i + kStep, p.V);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (now.at(j) > top) top = now.at(j), first = i + (j / E) * E * kThr + j % E;
      i += kStep;
    }
    float all = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    first = __reduce_min_sync(0xffffffffu, top == all ? first : 0x7fffffff);
    if (lane == 0) red[warp] = make_float2(all, __int_as_float(first));
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarpsV; ++w) all = fmaxf(all, red[w].x);
      first = 0x7fffffff;
      for (int w = 0; w < kWarpsV; ++w)
        if (red[w].x == all) first = min(first, __float_as_int(red[w].y));
      *out = make_float2(all, __int_as_float(first));
    }
    return;
  }
  const Cheap c = make_cheap(t);
  Running r = {-CUDART_INF_F, 0.f};
  if (head > 0 && chunk == 0) {
    r.top = fminf(fmaxf(extra, -CUDART_INF_F), CUDART_MAX_NORMAL_F);
    r.sum = r.top > -CUDART_INF_F ? 1.f : 0.f;
  }
  for (int n = 0; n < p.batches; ++n) {
    now = next;
    if (n + 1 < p.batches) next.load(z, i + (n + 1) * kStep, p.V);
#pragma unroll
    for (int h = 0; h < kPer / 16; ++h) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = now.at(16 * h + j);
      r.add(c, v);
    }
  }
  float top = r.top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = warp_sum(r.sum * cheap_weight(c, r.top, top));
  if (lane == 0) red[warp] = make_float2(top, sum);
  __syncthreads();
  if (warp == 0) {
    const float2 m = lane < kWarpsV ? red[lane] : make_float2(-CUDART_INF_F, 0.f);
    top = m.x;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    sum = m.y * cheap_weight(c, m.x, top);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) *out = make_float2(top, sum);
  }
}

// Maximum and sum (greedy: lowest index) of a row from its chunks.  Whole warps.
__device__ __forceinline__ float2 join(const float2* part, int chunks, bool greedy, const Cheap& c) {
  const int lane = threadIdx.x & 31;
  float2 m[kMaxChunks / 32];
  float top = -CUDART_INF_F;
#pragma unroll
  for (int a = 0; a < kMaxChunks / 32; ++a) {
    m[a] = 32 * a + lane < chunks ? part[32 * a + lane] : make_float2(-CUDART_INF_F, 0.f);
    top = fmaxf(top, m[a].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (greedy) {
    int first = 0x7fffffff;
#pragma unroll
    for (int a = 0; a < kMaxChunks / 32; ++a)
      if (32 * a + lane < chunks && m[a].x == top) first = min(first, __float_as_int(m[a].y));
    return make_float2(top, __int_as_float(__reduce_min_sync(0xffffffffu, first)));
  }
  float sum = 0.f;
  const float ref = fmaxf(top, -CUDART_MAX_NORMAL_F);
#pragma unroll
  for (int a = 0; a < kMaxChunks / 32; ++a) sum += m[a].x > -CUDART_INF_F ? m[a].y * cheap_weight(c, m[a].x, ref) : 0.f;
  return make_float2(top, warp_sum(sum));
}

struct Shared {
  uint32_t eighth[8];              // q4w_weights.cuh
  uint32_t by_p[8], by_q[8];       // the same divided by the row's mass
  int shift_p, shift_q;
  u64 mass_p, mass_q;
  u64 red[kWarpsV];
  int last, cross, first;
  u64 before;
  double per_t, log_mass;
};

// A number as m 2^e, m with its top bit set (0: zero); products are cut off, 63 bits and more.
// (fp64 has a sixtieth of the fp32 rate.)
struct Num {
  u64 m;
  int e;
  __device__ __forceinline__ static Num of(u64 v, int e) {
    const int z = v ? __clzll(v) : 0;
    return {v << z, e - z};
  }
  __device__ __forceinline__ static Num of(float v) {   // v >= 0, a normal number or 0
    const uint32_t b = __float_as_uint(v);
    return of(b >> 23 ? (b & 0x7fffffu) | 0x800000u : 0ull, (int)(b >> 23) - 150);
  }
  __device__ __forceinline__ Num operator*(const Num& o) const { return of(__umul64hi(m, o.m), e + o.e + 64); }
  __device__ __forceinline__ bool operator<(const Num& o) const {
    return o.m != 0 && (m == 0 || e < o.e || (e == o.e && m < o.m));
  }
};
// A single element's weight (28 bits of it, down to 2^-128).
__device__ __forceinline__ Num weight_number(const uint32_t* eighth, const Scale& s, float z) {
  z = capped(s, z);
  const float q = eighths(s, z);
  if (!(q < (float)sample::kBins)) return {0, 0};
  float nf;
  const int n = whole(q, &nf);
  return Num::of((u64)mantissa(s, z, q, nf) * eighth[n & 7], -59 - (n >> 3));
}
// ln of a share, from the logit: scale and ln of the mass may be formed before the logit is known.
__device__ __forceinline__ float log_prob(float z, float top, double per_t, double log_mass) {
  return (float)(((double)fminf(z, top) - (double)top) * per_t - log_mass);
}

// Inclusive scan over the CTA; *total: the sum.
__device__ __forceinline__ u64 block_incl(u64 v, u64* red, u64* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  u64 before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarpsV; ++w) {
    if (w < warp) before += red[w];
    sum += red[w];
  }
  *total = sum;
  return v + before;
}
// Sum of the lanes' masses, each below 2^54.
__device__ __forceinline__ u64 lanes_sum(u64 v) {
  const u64 lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
  return lo + ((u64)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27)) << 27);
}

// Eight neighbouring logits from index i on, NaN behind the row.
template <typename T>
struct Row {
  const T* z;
  int V;
  bool vec;
  __device__ __forceinline__ Row(const T* row, int v) : z(row), V(v), vec((reinterpret_cast<uintptr_t>(row) & 15) == 0) {}
  __device__ __forceinline__ void load(int i, float (&v)[8]) const {
    if (vec && i + 8 <= V) {
      T e[8];
#pragma unroll
      for (int a = 0; a < (int)sizeof(e) / 16; ++a)
        reinterpret_cast<uint4*>(e)[a] = reinterpret_cast<const uint4*>(z + i)[a];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = as_float(e[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i + j < V ? as_float(z[i + j]) : CUDART_NAN_F;
    }
  }
  // f(g, the lane's logits) for a warp's segments g, the next one's in flight
  template <typename F>
  __device__ __forceinline__ void sweep(int g0, int g1, F f) const {
    const int lane = threadIdx.x & 31;
    float v[8], next[8];
    if (g0 < g1) load(g0 * kSeg + 8 * lane, next);
#pragma unroll 1
    for (int g = g0; g < g1; g += kWarpsV) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = next[j];
      if (g + kWarpsV < g1) load((g + kWarpsV) * kSeg + 8 * lane, next);
      f(g, v);
    }
  }
};

// Whether this CTA is the last of the `ctas` that share a row; what the others wrote before is
// visible then.
__device__ __forceinline__ bool last_of_row(Shared& sh, unsigned* done, int ctas) {
  __syncthreads();   // the CTA's writes come before its first thread's fence, and so before its count
  if (threadIdx.x == 0) {
    __threadfence();
    sh.last = atomicAdd(done, 1u) == (unsigned)ctas - 1u;
    __threadfence();
  }
  __syncthreads();
  return sh.last;
}

// The first index whose running mass exceeds u times the whole, from the segments' masses;
// masses(i, w, v): those of the eight indices from i on, and their logits; logs(whole): by one
// thread, while the others search, and found(index, logit) after it.  False: no mass.
template <typename M, typename L, typename F>
__device__ __forceinline__ bool draw(const Params& p, Shared& sh, const u64* seg, float u, M masses, L logs, F found) {
  const int lane = threadIdx.x & 31;
  const int per = (p.n_segs + kThr - 1) / kThr, g0 = min((int)threadIdx.x * per, p.n_segs), g1 = min(g0 + per, p.n_segs);
  constexpr int kPer = (1 << 20) / kSeg / kThr;   // at most
  u64 m[kPer], sum = 0, total;
#pragma unroll
  for (int j = 0; j < kPer; ++j) m[j] = g0 + j < g1 ? __ldcg(seg + g0 + j) : 0ull;
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum += m[j];
  u64 run = block_incl(sum, sh.red, &total) - sum;
  if (total == 0) return false;
  const u64 goal = min(times(total, u, false), total - 1);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (run <= goal && run + m[j] > goal) sh.cross = g0 + j, sh.before = run;
    run += m[j];
  }
  __syncthreads();
  int at = -1;
  float logit = 0.f;
  if (threadIdx.x < 32) {
    const int i = sh.cross * kSeg + 8 * lane;
    u64 w[8];
    float v[8];
    masses(i, w, v);
    sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += w[j];
    u64 incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 a = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += a;
    }
    run = sh.before + incl - sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (run <= goal && run + w[j] > goal) at = i + j, logit = v[j];
      run += w[j];
    }
  } else if (threadIdx.x == 32) {
    logs(total);
  }
  __syncthreads();
  if (at >= 0) found(at, logit);
  return true;
}

// The part of the line of all units' segments that a CTA takes: at least one segment a warp.
struct Slice {
  int per, from, to;   // segments of a CTA; this one's first, and behind its last
  __device__ __forceinline__ Slice(const Params& p, int units) {
    const int all = units * p.n_segs;
    per = (max(kWarpsV, (all + p.ctas - 1) / p.ctas) + kWarpsV - 1) / kWarpsV * kWarpsV;
    from = (int)min((long long)blockIdx.x * per, (long long)all);
    to = min(from + per, all);
  }
  // CTAs that share unit i
  __device__ __forceinline__ int sharing(int n_segs, int i) const { return ((i + 1) * n_segs - 1) / per - i * n_segs / per + 1; }
};

__device__ __forceinline__ float random_of(const Params& p, int user, int j) {
  return fminf(fmaxf(p.u[(long long)user * (p.k + 1) + j], 0.f), 0.99999994f);
}

// Which of a user's drafts stand, and where the next token comes from.  Whole CTAs.
struct Chosen {
  float2 rows[2 * kMaxDrafts + 1];   // maximum and sum (greedy: lowest index)
  Unit unit;
};
template <typename T>
__device__ __forceinline__ void choose(const Params& p, int user, const uint32_t* eighth, Chosen& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.k;
  const float t = temperature_of(p, user);
  const bool greedy = t == 0.f;
  const int32_t* x = p.x + (long long)user * k;
  const int held = drafts_of(p, user);
  // what the first warp needs of the drafts, while the others join the rows
  constexpr int kTurns = kMaxDrafts / 32;
  float zx[kTurns], yx[kTurns], u[kTurns];
  int xs[kTurns];
  if (warp == 0) {
#pragma unroll
    for (int a = 0; a < kTurns; ++a) {
      const int j = 32 * a + lane;
      const bool here = j < held;
      xs[a] = here ? x[j] : -1;
      u[a] = here ? random_of(p, user, j) : 0.f;
      zx[a] = here ? as_float(row_of<T>(p, user, j)[xs[a]]) : 0.f;
      yx[a] = here && p.y ? as_float(row_of<T>(p, user, k + 1 + j)[xs[a]]) : 0.f;
    }
  }
  const Cheap cheap = make_cheap(greedy ? 1.f : t);
  for (int r = warp; r < (p.y ? 2 * k + 1 : k + 1); r += kWarpsV)
    if (needed(p, r, held, greedy)) {
      const float2 m = join(p.rows + ((long long)user * (2 * k + 1) + r) * p.chunks, p.chunks, greedy, cheap);
      if (lane == 0) sh.rows[r] = m;
    }
  __syncthreads();
  if (warp == 0) {
    int n = held;   // the first draft that falls, or `held`
#pragma unroll
    for (int a = 0; a < kTurns; ++a) {
      const int j = 32 * a + lane;
      bool stands = true;
      if (j < held) {
        const float2 rp = sh.rows[j];
        if (greedy) {
          stands = rp.x > -CUDART_INF_F && xs[a] == __float_as_int(rp.y);
        } else if (!(rp.x > -CUDART_INF_F)) {
          stands = false;
        } else {
          Num wq = Num::of(u[a]) * Num::of(rp.y), wp = weight_number(eighth, make_scale(rp.x, t, 0.f), zx[a]);
          if (p.y) {
            const float2 rq = sh.rows[k + 1 + j];
            if (rq.x > -CUDART_INF_F) {
              wq = wq * weight_number(eighth, make_scale(rq.x, t, 0.f), yx[a]);
              wp = wp * Num::of(rq.y);
            } else {
              wq = {0, 0};
            }
          }
          stands = wq < wp;
        }
      }
      const uint32_t falls = __ballot_sync(0xffffffffu, !stands);
      if (falls) {
        n = 32 * a + __ffs(falls) - 1;
        break;
      }
    }
    if (lane == 0) {
      Unit c = {user, n, kTarget, -1, t, sh.rows[n].x, 0.f, 0};
      if (!(c.top > -CUDART_INF_F)) {
        c.kind = kNothing;
      } else if (greedy) {
        c.kind = kLargest;
      } else if (n < held && !p.y) {
        c.without = x[n];
      } else if (n < held && sh.rows[k + 1 + n].x > -CUDART_INF_F) {
        c.kind = kRest;
        c.top_q = sh.rows[k + 1 + n].x;
      }
      sh.unit = c;
    }
  }
  __syncthreads();
}
// A user's row or rows in a list whose entry `at` is free.
__device__ __forceinline__ void list_rows(Unit* list, int at, Unit c) {
  list[at] = c;
  if (c.kind != kRest) return;
  c.top = c.top_q, c.drafted = 1;
  list[at + 1] = c;
}
// What is known of the outputs: the drafts that stand, the largest, the places behind.  (The log
// probabilities of the drafts: sums_kernel.)
__device__ __forceinline__ void write_chosen(const Params& p, const Chosen& sh) {
  const int j = threadIdx.x, k = p.k, user = sh.unit.user, n = sh.unit.n, kind = sh.unit.kind;
  if (j == 0) p.accepted[user] = n;
  if (j > k || (j == n && kind >= kTarget)) return;
  const long long at = (long long)user * (k + 1) + j;
  p.tokens[at] = j < n ? p.x[(long long)user * k + j] : j == n && kind == kLargest ? __float_as_int(sh.rows[n].y) : -1;
  if (p.logprobs && j >= n) p.logprobs[at] = j == n && kind == kNothing ? -CUDART_INF_F : 0.f;
}
template <typename T>
__device__ __forceinline__ void write_log(const Params& p, int user, int j, float2 row) {
  const float t = temperature_of(p, user);
  const float z = as_float(row_of<T>(p, user, j)[p.x[(long long)user * p.k + j]]);
  p.logprobs[(long long)user * (p.k + 1) + j] = t == 0.f ? 0.f : log_prob(z, row.x, 1.0 / (double)t, log((double)row.y));
}

template <typename T>
__global__ void __launch_bounds__(kThr) choose_kernel(const __grid_constant__ Params p) {
  __shared__ Chosen sh;
  __shared__ uint32_t eighth[8];
  const int user = blockIdx.x;
  if (threadIdx.x < 8) eighth[threadIdx.x] = sample::kEighth[threadIdx.x];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  choose<T>(p, user, eighth, sh);
  const Unit c = sh.unit;
  if (threadIdx.x == 0 && c.kind >= kTarget) {
    list_rows(p.list, atomicAdd(p.units, c.kind == kRest ? 2 : 1), c);
    if (c.kind == kRest) p.rest[atomicAdd(p.units + 1, 1)] = c;
  }
  if ((int)threadIdx.x < c.n) p.joined[(long long)user * (p.k + 1) + threadIdx.x] = sh.rows[threadIdx.x];
  write_chosen(p, sh);
}

constexpr double kSumUnit = 2.2737367544323206e-13;   // 2^-42

// Masses of p_n's row: those of the eight indices from i on, without the index that is left out.
__device__ __forceinline__ void weigh_target(const Shared& sh, const Scale& s, int without, int i, const float (&v)[8], u64 (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const Pair m = mantissas(s, v[j], v[j + 1]);
    w[j] = sample::weight_of(sh.eighth, m.mant[0], m.n[0]), w[j + 1] = sample::weight_of(sh.eighth, m.mant[1], m.n[1]);
  }
  if ((unsigned)(without - i) < 8u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = i + j != without ? w[j] : 0ull;
  }
}
// The draw from p_n alone, wherever it is made: by the segments' masses of weigh_target(), and with u = 0
// the first index that weighs anything, be it less than a unit.  False: nothing does.
template <typename T, typename L, typename F>
__device__ __forceinline__ bool draw_target(const Params& p, Shared& sh, const Row<T>& row, const Scale& s, int without, const u64* seg, float u,
                                            L logs, F found) {
  if (u != 0.f)
    return draw(p, sh, seg, u, [&](int i, u64 (&w)[8], float (&v)[8]) {
      row.load(i, v);
      weigh_target(sh, s, without, i, v, w);
    }, logs, found);
  u64 mass = 0;
  for (int g = threadIdx.x; g < p.n_segs; g += kThr) mass += __ldcg(seg + g);
  block_incl(mass, sh.red, &mass);
  if (threadIdx.x == 0) sh.first = 0x7fffffff, logs(mass);
  __syncthreads();
  for (int i0 = 0; i0 < p.V; i0 += kThr) {
    const int i = i0 + threadIdx.x;
    const bool some = i < p.V && i != without && eighths(s, capped(s, as_float(row.z[i]))) < (float)sample::kBins;
    if (some) atomicMin(&sh.first, i);
    if (__syncthreads_or(some)) break;
  }
  if (sh.first == 0x7fffffff) return false;
  if (threadIdx.x == 0) found(sh.first, as_float(row.z[sh.first]));
  return true;
}

// Exact masses of the listed rows, and the tokens that are drawn from p_n alone.  The CTAs behind
// the first p.ctas form the log probabilities of the drafts that stand.
// FEW: there was no choose_kernel, every CTA chooses for all of the few users.  (One user of four
// drafts from Python 26.8 us, with the kernel 29.9; from a graph 19.1 and 18.9.)
template <typename T, bool FEW>
__global__ void __launch_bounds__(kThr, kResident) sums_kernel(const __grid_constant__ Params p) {
  __shared__ Shared sh;
  __shared__ Chosen chosen[1];
  __shared__ Unit units[FEW ? 2 * kFewUsers : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.k;
  if (threadIdx.x < 8) sh.eighth[threadIdx.x] = sample::kEighth[threadIdx.x];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const bool logs_only = (int)blockIdx.x >= p.ctas;
  int n_units = 0;
  if constexpr (FEW) {
    int n_rest = 0;
    for (int user = 0; user < p.b; ++user) {
      choose<T>(p, user, sh.eighth, chosen[0]);
      const Unit c = chosen[0].unit;
      if (logs_only) {
        if ((int)threadIdx.x < c.n) write_log<T>(p, user, threadIdx.x, chosen[0].rows[threadIdx.x]);
      } else {
        if (threadIdx.x == 0 && c.kind >= kTarget) list_rows(units, n_units, c);
        if (blockIdx.x == 0) {
          if (threadIdx.x == 0 && c.kind == kRest) p.rest[n_rest] = c;
          write_chosen(p, chosen[0]);
        }
        n_units += c.kind == kRest ? 2 : c.kind == kTarget ? 1 : 0;
        n_rest += c.kind == kRest ? 1 : 0;
      }
      __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.units[1] = n_rest;
    if (logs_only) return;
  } else {
    if (logs_only) {
      const long long i = (long long)(blockIdx.x - p.ctas) * kThr + threadIdx.x;
      const int user = (int)(i / k), j = (int)(i % k);
      if (user < p.b && j < p.accepted[user]) write_log<T>(p, user, j, p.joined[(long long)user * (k + 1) + j]);
      return;
    }
    n_units = p.units[0];
  }
  const Slice slice(p, n_units);
  for (int at = slice.from; at < slice.to;) {
    const int unit = at / p.n_segs, first = at - unit * p.n_segs, g1 = min(p.n_segs, first + slice.to - at);
    at += g1 - first;
    const Unit c = FEW ? units[unit] : p.list[unit];
    const int user = c.user, n = c.n, without = c.without;
    const Scale s = make_scale(c.top, c.t, 0.f);
    const Row<T> row(row_of<T>(p, user, c.drafted ? k + 1 + n : n), p.V);
    u64* seg = p.seg + (long long)user * 2 * p.n_segs;
    u64 mine = 0;
    row.sweep(first + warp, g1, [&](int g, const float (&v)[8]) {
      u64 w[8], sum = 0;
      weigh_target(sh, s, without, g * kSeg + 8 * lane, v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += w[j];
      sum = lanes_sum(sum);
      if (lane == 0 && !c.drafted) seg[g] = sum;
      mine += sum;
    });
    if (c.kind == kRest) {
      if (lane == 0 && mine) atomicAdd(p.mass + 2 * user + c.drafted, mine);
      continue;
    }
    if (!last_of_row(sh, p.done + 2 * user, slice.sharing(p.n_segs, unit))) continue;
    auto logs = [&](u64 mass) {
      if (!p.logprobs) return;
      if (without >= 0) mass += weight(sh.eighth, s, capped(s, as_float(row.z[without])));   // of all of p_n
      sh.per_t = 1.0 / (double)c.t;
      sh.log_mass = log((double)mass * kSumUnit);
    };
    auto found = [&](int i, float z) {
      p.tokens[(long long)user * (k + 1) + n] = i;
      if (p.logprobs) p.logprobs[(long long)user * (k + 1) + n] = log_prob(z, c.top, sh.per_t, sh.log_mass);
    };
    const bool drawn = draw_target<T>(p, sh, row, s, without, seg, random_of(p, user, k), logs, found);
    // nothing but x_n weighs anything
    if (!drawn && threadIdx.x == 0) logs(0ull), found(without, as_float(row.z[without]));
    __syncthreads();
  }
}

// 2^(-j/8) / mass in 32 bits, times 2^(32 + *shift): mass in units of 2^-42, at least one.
// By one step of Newton's iteration from an fp32 quotient: 43 bits.
__device__ __forceinline__ void divide_table(u64 mass, const uint32_t* eighth, uint32_t* by, int* shift, int j) {
  const int c = __clzll(mass);
  const u64 m = mass << c;                                                    // [2^63, 2^64)
  const u64 r = (u64)(1.f / ((float)(uint32_t)(m >> 40) * 5.9604645e-08f) * 2147483648.f);   // near 2^95 / m
  const u64 near = __umul64hi(m, r) << 32 | (m * r) >> 32;                    // m r / 2^32, near 2^63
  const long long off = (long long)((1ull << 63) - near);
  const u64 quotient = (r << 31) + (u64)(((off >> 10) * (long long)r) >> 22);   // 2^126 / m
  by[j] = (uint32_t)min(__umul64hi(quotient, (u64)eighth[j] << 32) >> 30, 0xffffffffull);
  if (j == 0) *shift = 21 - c + 60 - kUnit;
}

// The two ends of a rest that masses do not decide, each a function: the kernel does not carry their code in line.
// The user's next token is i, of logit z.
__device__ __forceinline__ void write_drawn(const Params& p, const Shared& sh, const Unit& c, int i, float z) {
  const long long at = (long long)c.user * (p.k + 1) + c.n;
  p.tokens[at] = i;
  if (p.logprobs) p.logprobs[at] = log_prob(z, c.top, 1.0 / (double)c.t, log((double)sh.mass_p * kSumUnit));
}
// u = 0: the first index with p_n > q_n, be the difference less than a unit.  False: there is none.
template <typename T>
static __device__ __noinline__ bool rest_first(const Params& p, Shared& sh, int unit) {
  const Unit c = p.rest[unit];
  const T *zp = row_of<T>(p, c.user, c.n), *zq = row_of<T>(p, c.user, p.k + 1 + c.n);
  const Scale sp = make_scale(c.top, c.t, 0.f), sq = make_scale(c.top_q, c.t, 0.f);
  const Num mass_p = Num::of(sh.mass_p, 0), mass_q = Num::of(p.mass[2 * c.user + 1], 0);
  if (threadIdx.x == 0) sh.first = 0x7fffffff;
  __syncthreads();
  for (int i0 = 0; i0 < p.V; i0 += kThr) {
    const int i = i0 + threadIdx.x;
    const bool some = i < p.V && weight_number(sh.eighth, sq, as_float(zq[i])) * mass_p < weight_number(sh.eighth, sp, as_float(zp[i])) * mass_q;
    if (some) atomicMin(&sh.first, i);
    if (__syncthreads_or(some)) break;
  }
  if (sh.first == 0x7fffffff) return false;
  if (threadIdx.x == 0) write_drawn(p, sh, c, sh.first, as_float(zp[sh.first]));
  return true;
}
// The rest is empty: from p_n.
template <typename T>
static __device__ __noinline__ void rest_from_target(const Params& p, Shared& sh, int unit) {
  const Unit c = p.rest[unit];
  auto logs = [](u64) {};   // write_drawn() forms them
  auto found = [&](int i, float z) { write_drawn(p, sh, c, i, z); };
  __syncthreads();
  draw_target<T>(p, sh, Row<T>(row_of<T>(p, c.user, c.n), p.V), make_scale(c.top, c.t, 0.f), -1,
                 p.seg + (long long)c.user * 2 * p.n_segs, random_of(p, c.user, p.k), logs, found);
}

// Masses of the rest, max(p_n - q_n, 0), and the tokens drawn from it.
template <typename T>
__global__ void __launch_bounds__(kThr, kResident) rest_kernel(const __grid_constant__ Params p) {
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 8) sh.eighth[threadIdx.x] = sample::kEighth[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  const Slice slice(p, p.units[1]);
  for (int at = slice.from; at < slice.to;) {
    const int unit = at / p.n_segs, first = at - unit * p.n_segs, g1 = min(p.n_segs, first + slice.to - at);
    at += g1 - first;
    const Unit c = p.rest[unit];
    const int user = c.user;
    const Row<T> rp(row_of<T>(p, user, c.n), p.V), rq(row_of<T>(p, user, p.k + 1 + c.n), p.V);
    float vn[8], yn[8];
    if (first + warp < g1) rp.load((first + warp) * kSeg + 8 * lane, vn), rq.load((first + warp) * kSeg + 8 * lane, yn);
    __syncthreads();
    if (threadIdx.x < 16) {
      const bool q = threadIdx.x >= 8;
      const u64 mass = p.mass[2 * user + q];
      if (!q) sh.mass_p = mass;
      divide_table(mass, sh.eighth, q ? sh.by_q : sh.by_p, q ? &sh.shift_q : &sh.shift_p, threadIdx.x & 7);
    }
    __syncthreads();
    const Scale sp = make_scale(c.top, c.t, 0.f), sq = make_scale(c.top_q, c.t, 0.f);
    // probabilities in units of 2^-53
    auto probabilities = [](const uint32_t* by, int shift, const Scale& s, float z0, float z1, u64 (&w)[2]) {
      const Pair m = mantissas(s, z0, z1);
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = shift_right((u64)m.mant[i] * by[m.n[i] & 7], shift + (m.n[i] >> 3));
    };
    auto weigh = [&](const float (&v)[8], const float (&y)[8], u64 (&w)[8]) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        u64 a[2], b[2];
        probabilities(sh.by_p, sh.shift_p, sp, v[j], v[j + 1], a);
        probabilities(sh.by_q, sh.shift_q, sq, y[j], y[j + 1], b);
#pragma unroll
        for (int i = 0; i < 2; ++i) w[j + i] = a[i] > b[i] ? a[i] - b[i] : 0ull;
      }
    };
    u64* seg = p.seg + ((long long)user * 2 + 1) * p.n_segs;
#pragma unroll 1
    for (int g = first + warp; g < g1; g += kWarpsV) {
      float v[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = vn[j], y[j] = yn[j];
      if (g + kWarpsV < g1) rp.load((g + kWarpsV) * kSeg + 8 * lane, vn), rq.load((g + kWarpsV) * kSeg + 8 * lane, yn);
      u64 w[8], sum = 0;
      weigh(v, y, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += w[j];
      sum = lanes_sum(sum);
      if (lane == 0) seg[g] = sum;
    }
    if (!last_of_row(sh, p.done + 2 * user + 1, slice.sharing(p.n_segs, unit))) continue;
    auto logs = [&](u64) {
      sh.per_t = 1.0 / (double)c.t;
      sh.log_mass = log((double)sh.mass_p * kSumUnit);
    };
    auto found = [&](int i, float z) {
      p.tokens[(long long)user * (p.k + 1) + c.n] = i;
      if (p.logprobs) p.logprobs[(long long)user * (p.k + 1) + c.n] = log_prob(z, c.top, sh.per_t, sh.log_mass);
    };
    const float u = random_of(p, user, p.k);
    const bool drawn = u == 0.f ? rest_first<T>(p, sh, unit) : draw(p, sh, seg, u, [&](int i, u64 (&w)[8], float (&v)[8]) {
      float y[8];
      rp.load(i, v);
      rq.load(i, y);
      weigh(v, y, w);
    }, logs, found);
    if (!drawn) rest_from_target<T>(p, sh, unit);   // the two are one
  }
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

static void sizes(int b, int k, int V, size_t (&at)[9]) {
  const size_t users = (size_t)b, chunks = min((size_t)kMaxChunks, ((size_t)V + 4095) / 4096), segs = ((size_t)V + kSeg - 1) / kSeg;
  const size_t bytes[8] = {users * (2 * (size_t)k + 1) * chunks * sizeof(float2), users * ((size_t)k + 1) * sizeof(float2), 2 * sizeof(int),
                           2 * users * sizeof(Unit), users * sizeof(Unit), 2 * users * sizeof(u64), users * 2 * segs * sizeof(u64),
                           2 * users * sizeof(unsigned)};
  at[0] = 0;
  for (int i = 0; i < 8; ++i) at[i + 1] = at[i] + up256(bytes[i]);
}

template <typename T>
static int launch(const Params& p, int b, cudaStream_t s) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThr);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.chunks, p.y ? 2 * p.k + 1 : p.k + 1, b);
  cudaError_t e = cudaLaunchKernelEx(&cfg, rows_kernel<T>, p);
  const bool few = b <= kFewUsers;
  if (!few) {
    cfg.gridDim = dim3(b);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, choose_kernel<T>, p);
  }
  const unsigned logs = !p.logprobs || p.k == 0 ? 0 : few ? 1 : (unsigned)(((long long)b * p.k + kThr - 1) / kThr);
  cfg.gridDim = dim3(p.ctas + logs);
  if (e == cudaSuccess) e = few ? cudaLaunchKernelEx(&cfg, sums_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, sums_kernel<T, false>, p);
  cfg.gridDim = dim3(p.ctas);
  if (e == cudaSuccess && p.y) e = cudaLaunchKernelEx(&cfg, rest_kernel<T>, p);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "draft verification launch");
}

}  // namespace verify

size_t draft_verify_bytes(int b, int k, int V) {
  size_t at[9];
  verify::sizes(b, k, V, at);
  return at[8];
}

int launch_draft_verify(const DraftVerify& d, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  using namespace verify;
  size_t at[9];
  sizes(d.b, d.k, d.V, at);
  char* w = static_cast<char*>(ws);
  // of the first kernel: enough CTAs for several rounds of the card, more batches each beyond
  const int step = kThr * 64 / (d.dtype == Q4_F32 ? 4 : 2), n = (d.V + step - 1) / step;
  const long long all = (long long)d.b * (2 * d.k + 1) * n;
  const int batches = max((n + kMaxChunks - 1) / kMaxChunks, (int)min((long long)kMaxBatches, all / (dev.sms * kRowCtas)));
  const Params p = {d.logits, d.draft_logits, d.user_stride, d.row_stride, d.draft_user_stride, d.draft_row_stride, d.drafts, d.u,
                    d.temperature, d.tokens, d.accepted, d.logprobs, d.b, d.k, d.V, (n + batches - 1) / batches, batches,
                    (d.V + kSeg - 1) / kSeg, dev.sms * kResident, reinterpret_cast<float2*>(w + at[0]), reinterpret_cast<float2*>(w + at[1]),
                    reinterpret_cast<int*>(w + at[2]), reinterpret_cast<Unit*>(w + at[3]), reinterpret_cast<Unit*>(w + at[4]),
                    reinterpret_cast<u64*>(w + at[5]), reinterpret_cast<u64*>(w + at[6]), reinterpret_cast<unsigned*>(w + at[7])};
  return d.dtype == Q4_F32 ? launch<float>(p, d.b, s) : d.dtype == Q4_F16 ? launch<__half>(p, d.b, s) : launch<__nv_bfloat16>(p, d.b, s);
}

}  // namespace q4w
