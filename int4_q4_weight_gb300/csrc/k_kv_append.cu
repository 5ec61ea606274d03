// Appending the keys and values of new tokens to a paged cache, the position
// rotation applied on the way, and the queries rotated in the same pass.
//
// Token t, the j-th of the n new tokens of its sequence, takes cache position
// P = kv_len - n + j.  With the rotary position p (P, or positions[t]) and
// steps_i turns per position in units of 2^-64, pair i turns by
// a_i = 2 pi frac(p steps_i 2^-64):  (x, y) -> (x cos a - y sin a,
// y cos a + x sin a).  The product p * steps_i wraps modulo 2^64, which is
// the reduction of the angle by whole turns without any rounding: far
// positions keep the full precision (the error is p * 2^-65 turns from the
// rounding of the step), where an fp32 angle at p = 10^6 is off by 0.06 rad.
//
// Bound: HBM (every input element is read and every output written once); at
// decode sizes the launch.  A thread owns 16 elements of a row (eight pairs):
// the eight sines and cosines are formed once and used for every row (head)
// of the token that the thread takes.  The rows are loaded one ahead, the first
// before the position is looked up: those lookups are three loads one after the
// other, and while they run nothing else would be in flight.
//
// Two more forms of the same pass: with a norm of each head before the rotation,
//   y = x rsqrt(mean x^2 + eps) w   (fp32, the D / 16 threads of a row sum by shuffles; a row whose
//   squares leave fp32 is summed again, scaled by a power of two),
// and, after it, into a cache of int8 codes with a scale per 32 elements: the scale is the
// block's largest magnitude / 127, rounded up to fp16, so that no code is cut off and a
// value is half a scale off at most; a thread's two runs of eight lie in one block each,
// whose four maxima meet in shared memory.
//
// Measured: 16 ragged prompts, 41000 tokens of 8 + 2 rows of 256, bf16 (421 MB):
// 75 us, 5.6 TB/s, half of it writes.  Blocks of 128 threads so that few finish
// late; more resident blocks, or two rows ahead, were slower.  8 tokens: 3.2 us.
// With norms: 8 ragged prompts, 21000 tokens of 16 + 16 heads of 128, bf16 (348 MB): 71 us, 4.9 TB/s
// (78 before norms and rotation took two elements an instruction: 20 of them an element, issue active for
// 64 % of the cycles); f32 (522 MB) 87 us, 6.0 TB/s.  Quantised: 8 prompts of 8 + 2 heads of 256, bf16 (207 MB)
// 54 us, 3.8 TB/s, 22 instructions an element; f32 (316 MB) 68 us, 4.6.
#include <type_traits>

#include "q4w_codes.cuh"
#include "q4w_device.cuh"
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"

namespace q4w {
namespace append {

constexpr int kThr = 128;
constexpr int kChunk = 16;   // elements of a row per thread: eight pairs

enum Mode { kPlain, kNorm, kQ8 };   // kQ8: with norms where they are given

struct Params {
  KvTables kv;
  const void *k, *v, *q;                     // [T][heads][D], token strides in elements
  long long k_stride, v_stride, q_stride;
  void *k_cache, *v_cache, *q_out;           // cache type
  const uint64_t* steps;                     // [rot / 2]
  const int32_t* positions;                  // [T] or NULL
  int32_t* err;
  int T, D, n_q, rot, interleaved;
  int rows, groups, rows_per_group;          // rows: n_q + 2 n_kv heads of a token
  // the norms (kNorm, kQ8): weights [D] or NULL; the scales of the caches (kQ8), which hold codes
  const float *q_norm, *k_norm, *v_norm;
  float eps, inv_d;                          // 1 / D, a power of two
  __half *k_scales, *v_scales;
};

// 16 bytes of an input.  It is the output of the kernel before, which may still be
// writing when this one starts: not the non-coherent load, and ordered (volatile, with
// the clobber) behind the wait for that kernel.  The loads of the next row stand
// before the stores of the last one in the source, so they need no freedom to pass them.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// Eight consecutive elements, as loaded and as fp32.
template <typename IN>
struct Eight {
  uint4 w[sizeof(IN) / 2];
  __device__ __forceinline__ void load(const IN* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(IN) / 2; ++i) w[i] = ld16(p + 4 * i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t* u = &w[0].x;
    if constexpr (sizeof(IN) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Half16<IN>::unpack(u[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
};

template <typename OUT>
__device__ __forceinline__ void store8(OUT* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(Half16<OUT>::pack(x[0], x[1]), Half16<OUT>::pack(x[2], x[3]),
                                            Half16<OUT>::pack(x[4], x[5]), Half16<OUT>::pack(x[6], x[7]));
}

// Eight elements times f and their norm weights, from element i on.  The weights come from
// L1 for every row: held in registers (16) they cost a third of the resident threads.
__device__ __forceinline__ void scale8(float (&x)[8], float f, const float* w, int i) {
  const float4 u = *reinterpret_cast<const float4*>(w + i), v = *reinterpret_cast<const float4*>(w + i + 4);
  const float ws[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  const f2_t f2 = f2_pack(f, f);
#pragma unroll
  for (int k = 0; k < 8; k += 2) f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), f2_mul(f2, f2_pack(ws[k], ws[k + 1]))), x[k], x[k + 1]);
}

// Where a mean of squares keeps its digits: what is lost below the normal numbers is 2^-40 of it, and
// the sum of 512 is finite.
constexpr float kLeastMean = 7.8886091e-31f, kMostMean = 1.3292280e36f;   // 2^-100, 2^120

constexpr float kMaxScale = 515.5f;   // 127 of it are a finite fp16 number, as the attention needs
// The largest magnitude as bits: a NaN's are above an infinity's.
__device__ __forceinline__ uint32_t top_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}
// Scale of a block by its largest magnitude: fp16 of top / 127, rounded up; 0, and `bad`, for
// a block that holds an infinity or NaN, or whose scale is above the largest.
__device__ __forceinline__ __half block_scale(uint32_t top, bool* bad) {
  const __half s = __float2half_ru(__fdiv_ru(__uint_as_float(top), 127.f));
  *bad = top >= 0x7f800000u || __half2float(s) > kMaxScale;
  return *bad ? __half(0.f) : s;
}
// Eight codes of x / scale.  y + 1.5 * 2^23 has the nearest integer in its lowest bits; the
// product is rounded first, so that most exact halves (16-bit inputs have many) stay halves.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], __half scale) {
  const float s = __half2float(scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = s > 0.f ? __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.f)) : 0u;
  auto four = [&](int i) { return __byte_perm(__byte_perm(u[i], u[i + 1], 0x0040), __byte_perm(u[i + 2], u[i + 3], 0x0040), 0x5410); };
  return make_uint2(four(0), four(4));
}

// Resident blocks: with norms seven (72 registers, 8 bytes of spills for fp16 input).  Eight ragged prompts of
// 16 + 16 heads of 128, bf16 | fp16 | f32 input, us: five 71 | 78 | 93, six 73 | 72.5 | 86, seven 71.5 | 72 | 87,
// eight 74.5 | 79 | 118.  Quantised six (80 registers, 4 bytes of spills for fp16, 36 for f32); eight prompts of
// 8 + 2 heads of 256: five 59 | 58 | 68, six 54 | 54 | 68, seven 57 | 56 | 84, eight 65 | 65 | 93.
template <typename IN, typename OUT, int MODE>
__global__ void __launch_bounds__(kThr, MODE == kPlain ? 0 : MODE == kNorm ? 7 : 6) append_kernel(const __grid_constant__ Params p) {
  __shared__ int first_sh;
  __shared__ __align__(16) uint32_t top_sh[MODE == kQ8 ? 2 : 1][MODE == kQ8 ? 2 * kThr : 4];   // by the row's parity
  pdl_wait();
  const int chunks = p.D / kChunk;
  const long long idx = (long long)blockIdx.x * kThr + threadIdx.x;
  const int c = (int)(idx % chunks);
  const long long tg = idx / chunks;
  const int grp = (int)(tg % p.groups);
  const int tok = (int)min(tg / p.groups, (long long)p.T);   // T: past the end
  // where the thread's two halves of eight elements lie in a row
  const bool rotates = c < p.rot / kChunk;
  const int lo = rotates && !p.interleaved ? c * 8 : c * kChunk;
  const int hi = rotates && !p.interleaved ? lo + p.rot / 2 : lo + 8;
  const int r0 = grp * p.rows_per_group, r1 = min(r0 + p.rows_per_group, p.rows);
  auto source = [&](int r) {
    if (r < p.n_q) return static_cast<const IN*>(p.q) + tok * p.q_stride + (long long)r * p.D;
    r -= p.n_q;
    if (r < p.kv.n_kv) return static_cast<const IN*>(p.k) + tok * p.k_stride + (long long)r * p.D;
    return static_cast<const IN*>(p.v) + tok * p.v_stride + (long long)(r - p.kv.n_kv) * p.D;
  };
  Eight<IN> na, nb;   // the next row's
  const IN* src = nullptr;
  if (tok < p.T) {
    src = source(r0);
    na.load(src + lo);
    nb.load(src + hi);
  }
  // the sequence of this block's first token: how many sequences end at or
  // before it (counted by all threads; a thread's own token is a few further)
  if (threadIdx.x == 0) first_sh = 0;
  __syncthreads();
  {
    const int t0 = (int)((long long)blockIdx.x * kThr / chunks / p.groups);
    int n = 0;
    for (int i = threadIdx.x; i < p.kv.n_seqs; i += kThr) n += p.kv.cu_tokens[i + 1] <= t0;
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&first_sh, n);
  }
  __syncthreads();
  if (tok >= p.T) return;
  int seq = first_sh;
  while (seq < p.kv.n_seqs && p.kv.cu_tokens[seq + 1] <= tok) ++seq;
  if (seq >= p.kv.n_seqs) return;   // a padding token behind the last sequence

  const int pos = p.kv.kv_lens[seq] - p.kv.cu_tokens[seq + 1] + tok;
  const int page = kv_page(p.kv, seq, pos);
  const bool stored = page >= 0;
  if (!stored && c == 0 && p.err) *p.err = 1;

  float cs[8], sn[8];
  if (rotates) {
    const long long at = p.positions ? p.positions[tok] : pos;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t phase = (uint64_t)at * p.steps[c * 8 + i];
      // the upper 32 bits as a signed fraction of a half turn
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);
    }
  }

  // the lanes of this row: 4 to 32, side by side, and all on the same path
  const int lane = threadIdx.x & 31;
  const uint32_t peers = chunks == 32 ? 0xffffffffu : ((1u << chunks) - 1u) << (lane & ~(chunks - 1));
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    float a[8], b[8];
    na.get(a);
    nb.get(b);
    if (r + 1 < r1) {   // the heads of a token lie side by side
      src = r + 1 == p.n_q || r + 1 == p.n_q + p.kv.n_kv ? source(r + 1) : src + p.D;
      na.load(src + lo);
      nb.load(src + hi);
    }
    OUT* dst;
    long long row = 0;
    const bool is_q = r < p.n_q, is_k = !is_q && r < p.n_q + p.kv.n_kv;
    if (is_q) {
      dst = static_cast<OUT*>(p.q_out) + ((long long)tok * p.n_q + r) * p.D;
    } else {
      if (!stored) continue;
      const int h = is_k ? r - p.n_q : r - p.n_q - p.kv.n_kv;
      row = kv_row(p.kv, page, h) + pos % p.kv.page_size;
      dst = static_cast<OUT*>(is_k ? p.k_cache : p.v_cache) + row * p.D;   // kQ8: not used
    }
    if constexpr (MODE != kPlain) {
      const float* w = is_q ? p.q_norm : is_k ? p.k_norm : p.v_norm;
      if (w) {
        // (fp16 input: its squares, from 2^-48 to 2^32, need no second turn)
        float eps = p.eps, mean;
#pragma unroll 1
        for (bool again = std::is_same<IN, __half>::value;; again = true) {
          f2_t sums = f2_pack(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const f2_t x = f2_pack(a[i], a[i + 1]), y = f2_pack(b[i], b[i + 1]);
            sums = f2_fma(x, x, f2_fma(y, y, sums));
          }
          float sum, odd;
          f2_unpack(sums, sum, odd);
          sum += odd;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            if (chunks > o) sum += __shfl_xor_sync(peers, sum, o);
          mean = fmaf(sum, p.inv_d, eps);
          if (again || (mean >= kLeastMean && mean <= kMostMean)) break;
          // Once more, the row and the root of eps times a power of two that leaves the larger of them in
          // [1, 2).  (The lanes of a row have the same sum, bit for bit.)
          uint32_t top = max(top_bits(a), top_bits(b));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            if (chunks > o) top = max(top, __shfl_xor_sync(peers, top, o));
          int e = (int)(top >> 23) - 127;
          if (eps > 0.f) e = max(e, ((int)(__float_as_uint(eps) >> 23) - 127) >> 1);
          const float by = __uint_as_float((uint32_t)(127 - min(max(e, -126), 126)) << 23);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= by, b[i] *= by;
          eps = eps * by * by;
        }
        const float f = rsqrtf(mean);
        scale8(a, f, w, lo);
        scale8(b, f, w, hi);
      }
    }
    if (rotates && (is_q || is_k)) {
      if (p.interleaved) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = a[i], x[8 + i] = b[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = x[2 * i], o = x[2 * i + 1];
          x[2 * i] = fmaf(e, cs[i], -o * sn[i]);
          x[2 * i + 1] = fmaf(o, cs[i], e * sn[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = x[i], b[i] = x[8 + i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const f2_t e = f2_pack(a[i], a[i + 1]), o = f2_pack(b[i], b[i + 1]), c2 = f2_pack(cs[i], cs[i + 1]), s2 = f2_pack(sn[i], sn[i + 1]);
          const f2_t n2 = f2_pack(-sn[i], -sn[i + 1]);
          f2_unpack(f2_fma(e, c2, f2_mul(o, n2)), a[i], a[i + 1]);
          f2_unpack(f2_fma(o, c2, f2_mul(e, s2)), b[i], b[i + 1]);
        }
      }
    }
    if constexpr (MODE == kQ8) {
      if (!is_q) {
        uint32_t* const top = top_sh[r & 1] + 2 * (threadIdx.x & ~(chunks - 1));   // of the row's runs of eight
        top[lo >> 3] = top_bits(a);
        top[hi >> 3] = top_bits(b);
        __syncwarp(peers);
        const uint4 ta = *reinterpret_cast<const uint4*>(top + (lo >> 5) * 4), tb = *reinterpret_cast<const uint4*>(top + (hi >> 5) * 4);
        bool bad_a, bad_b;
        const __half sa = block_scale(max(max(ta.x, ta.y), max(ta.z, ta.w)), &bad_a);
        const __half sb = block_scale(max(max(tb.x, tb.y), max(tb.z, tb.w)), &bad_b);
        int8_t* codes = static_cast<int8_t*>(is_k ? p.k_cache : p.v_cache) + row * p.D;
        __half* scales = (is_k ? p.k_scales : p.v_scales) + row * (p.D / 32);
        *reinterpret_cast<uint2*>(codes + lo) = codes8(a, sa);
        *reinterpret_cast<uint2*>(codes + hi) = codes8(b, sb);
        if ((lo & 31) == 0) scales[lo >> 5] = sa;
        if ((hi & 31) == 0) scales[hi >> 5] = sb;
        if ((bad_a || bad_b) && p.err) *p.err = 1;
        continue;
      }
    }
    store8(dst + lo, a);
    store8(dst + hi, b);
  }
}

template <typename IN, typename OUT, int MODE>
static int launch(const Params& p, cudaStream_t s) {
  const long long n = (long long)p.T * p.groups * (p.D / kChunk);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + kThr - 1) / kThr));
  cfg.blockDim = dim3(kThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<IN, OUT, MODE>, p);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "KV append launch");
}

template <int MODE>
static int launch_mode(const Params& p, int in_dtype, bool f16, cudaStream_t s) {
  switch (in_dtype) {
    case Q4_F32: return f16 ? launch<float, __half, MODE>(p, s) : launch<float, __nv_bfloat16, MODE>(p, s);
    case Q4_F16: return f16 ? launch<__half, __half, MODE>(p, s) : launch<__half, __nv_bfloat16, MODE>(p, s);
    default: return f16 ? launch<__nv_bfloat16, __half, MODE>(p, s) : launch<__nv_bfloat16, __nv_bfloat16, MODE>(p, s);
  }
}

// Reading rows of a quantised cache back: value = code * scale, rounded once to OUT.
// A thread takes 16 codes of K and of V of a row; HBM, two thirds of it writes.  Codes
// are widened without the conversion unit (a quarter of the rate): to fp16 (q4w_codes.cuh), where
// one product is rounded to the output, or as the low byte of 2^23 to fp32.
// Four caches of up to 16384 rows of 512 (135 MB): 26.4 us, 5.1 TB/s; blocks of 256 threads 27.3,
// two or four places a thread 29.6 and 32.3.
struct ReadParams {
  KvTables kv;
  const int8_t *k, *v;
  const __half *k_scales, *v_scales;
  void *k_out, *v_out;
  int32_t* err;
  int T, D, lg_chunks;
};
constexpr int kReadThr = 128;

template <typename OUT>
__device__ __forceinline__ void widen16(const uint4 code, __half scale, OUT* out) {
  const uint32_t u[4] = {code.x ^ 0x80808080u, code.y ^ 0x80808080u, code.z ^ 0x80808080u, code.w ^ 0x80808080u};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<OUT, __half>::value) {
      const uint32_t lo = two_codes<0, 1>(u[i]), hi = two_codes<2, 3>(u[i]);
      const __half2 s = __half2half2(scale), a = __hmul2(*reinterpret_cast<const __half2*>(&lo), s), b = __hmul2(*reinterpret_cast<const __half2*>(&hi), s);
      r[2 * i] = *reinterpret_cast<const uint32_t*>(&a), r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const float s = __half2float(scale);
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = (__uint_as_float(__byte_perm(u[i], 0x4b000000u, 0x7540 | k)) - 8388736.f) * s;   // 2^23 + 128
      r[2 * i] = Half16<OUT>::pack(x[0], x[1]), r[2 * i + 1] = Half16<OUT>::pack(x[2], x[3]);
    }
  }
  reinterpret_cast<uint4*>(out)[0] = make_uint4(r[0], r[1], r[2], r[3]);
  reinterpret_cast<uint4*>(out)[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

template <typename OUT>
__global__ void __launch_bounds__(kReadThr) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_wait();
  const uint32_t per_tok = (uint32_t)p.kv.n_kv << p.lg_chunks;
  const long long idx0 = (long long)blockIdx.x * kReadThr;
  const int t0 = (int)(idx0 / per_tok);
  const uint32_t local = (uint32_t)(idx0 - (long long)t0 * per_tok) + threadIdx.x, ahead = local / per_tok, rest = local - ahead * per_tok;
  const long long tok = (long long)t0 + ahead;
  // the token's sequence: how many end at or before the warp's first token, then on
  const long long first = __shfl_sync(0xffffffffu, tok, 0);
  int seq = 0;
  for (int i = threadIdx.x & 31; i - (int)(threadIdx.x & 31) < p.kv.n_seqs; i += 32) {
    const uint32_t before = __ballot_sync(0xffffffffu, i < p.kv.n_seqs && p.kv.cu_tokens[i + 1] <= first);
    seq += __popc(before);
    if (before != 0xffffffffu) break;
  }
  if (tok >= p.T) return;
  int end = 0;
  while (seq < p.kv.n_seqs && (end = p.kv.cu_tokens[seq + 1]) <= tok) ++seq;
  if (seq >= p.kv.n_seqs) return;   // a padding token behind the last sequence
  const int pos = p.kv.kv_lens[seq] - end + (int)tok;
  const int page = kv_page(p.kv, seq, pos);
  if (page < 0 && p.err) *p.err = 1;
  const int h = (int)(rest >> p.lg_chunks), c = (int)(rest & ((1u << p.lg_chunks) - 1u));
  const long long at = (page < 0 ? 0 : kv_row(p.kv, page, h) + pos % p.kv.page_size) * p.D + c * kChunk;
  const long long to = (tok * p.kv.n_kv + h) * p.D + c * kChunk;
  uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
  __half ks = __half(0.f), vs = ks;
  if (page >= 0) {
    k = *reinterpret_cast<const uint4*>(p.k + at), v = *reinterpret_cast<const uint4*>(p.v + at);
    ks = p.k_scales[at >> 5], vs = p.v_scales[at >> 5];
  }
  widen16(k, ks, static_cast<OUT*>(p.k_out) + to);
  widen16(v, vs, static_cast<OUT*>(p.v_out) + to);
}

}  // namespace append

int launch_kv_append(const KvAppend& c, const DeviceInfo& dev, cudaStream_t s) {
  append::Params p = {};
  p.kv = kv_tables(c.cache);
  p.k = c.k, p.v = c.v, p.q = c.q;
  p.k_stride = c.k_stride, p.v_stride = c.v_stride, p.q_stride = c.q_stride;
  p.k_cache = c.cache.k, p.v_cache = c.cache.v, p.q_out = c.q_out;
  p.k_scales = reinterpret_cast<__half*>(c.k_scales), p.v_scales = reinterpret_cast<__half*>(c.v_scales);
  p.q_norm = c.q_norm, p.k_norm = c.k_norm, p.v_norm = c.v_norm;
  p.eps = c.eps, p.inv_d = 1.f / (float)c.cache.head_dim;
  p.steps = c.steps;
  p.positions = c.positions;
  p.err = c.err;
  p.T = c.T, p.D = c.cache.head_dim, p.n_q = c.n_q, p.rot = c.rot, p.interleaved = c.interleaved;
  p.rows = c.n_q + 2 * c.cache.n_kv;
  // Rows a thread takes: all of a token's while that still fills the device
  // (one set of sines per token and pair), else fewer, down to one.
  const long long want = (long long)dev.sms * 2048;   // resident threads of the device
  const long long per_row = (long long)c.T * (p.D / append::kChunk);
  int groups = (int)((want + per_row - 1) / per_row);
  if (groups > p.rows) groups = p.rows;
  p.rows_per_group = (p.rows + groups - 1) / groups;
  p.groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
  const bool f16 = c.cache.dtype == Q4_F16;
  if (c.k_scales) return append::launch_mode<append::kQ8>(p, c.in_dtype, f16, s);
  if (c.q_norm || c.k_norm || c.v_norm) return append::launch_mode<append::kNorm>(p, c.in_dtype, f16, s);
  return append::launch_mode<append::kPlain>(p, c.in_dtype, f16, s);
}

int launch_kv_read_q8(const q4_kv_cache_q8& c, int T, void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  append::ReadParams p = {};
  p.kv = kv_tables(c.c);
  p.k = static_cast<const int8_t*>(c.c.k), p.v = static_cast<const int8_t*>(c.c.v);
  p.k_scales = reinterpret_cast<const __half*>(c.k_scales), p.v_scales = reinterpret_cast<const __half*>(c.v_scales);
  p.k_out = k_out, p.v_out = v_out;
  p.err = err;
  p.T = T, p.D = c.c.head_dim;
  p.lg_chunks = p.D == 64 ? 2 : p.D == 128 ? 3 : p.D == 256 ? 4 : 5;
  const long long n = (long long)T * c.c.n_kv * (p.D / append::kChunk), per = append::kReadThr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + per - 1) / per));
  cfg.blockDim = dim3(append::kReadThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = c.c.dtype == Q4_F16 ? cudaLaunchKernelEx(&cfg, append::read_kernel<__half>, p)
                                            : cudaLaunchKernelEx(&cfg, append::read_kernel<__nv_bfloat16>, p);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "KV read launch");
}

}  // namespace q4w
