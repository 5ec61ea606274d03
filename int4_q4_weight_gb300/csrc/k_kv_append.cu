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
// Measured: 16 ragged prompts, 41000 tokens of 8 + 2 rows of 256, bf16 (421 MB):
// 75 us, 5.6 TB/s, half of it writes.  Blocks of 128 threads so that few finish
// late; more resident blocks, or two rows ahead, were slower.  8 tokens: 3.2 us.
#include "q4w_device.cuh"
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"

namespace q4w {
namespace append {

constexpr int kThr = 128;
constexpr int kChunk = 16;   // elements of a row per thread: eight pairs

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

template <typename IN, typename OUT>
__global__ void __launch_bounds__(kThr) append_kernel(const __grid_constant__ Params p) {
  __shared__ int first_sh;
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
  if (tok < p.T) {
    na.load(source(r0) + lo);
    nb.load(source(r0) + hi);
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

#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    float a[8], b[8];
    na.get(a);
    nb.get(b);
    if (r + 1 < r1) {
      na.load(source(r + 1) + lo);
      nb.load(source(r + 1) + hi);
    }
    OUT* dst;
    const bool is_q = r < p.n_q, is_k = !is_q && r < p.n_q + p.kv.n_kv;
    if (is_q) {
      dst = static_cast<OUT*>(p.q_out) + ((long long)tok * p.n_q + r) * p.D;
    } else {
      if (!stored) continue;
      const int h = is_k ? r - p.n_q : r - p.n_q - p.kv.n_kv;
      dst = static_cast<OUT*>(is_k ? p.k_cache : p.v_cache) + (kv_row(p.kv, page, h) + pos % p.kv.page_size) * p.D;
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
        for (int i = 0; i < 8; ++i) {
          const float e = a[i], o = b[i];
          a[i] = fmaf(e, cs[i], -o * sn[i]);
          b[i] = fmaf(o, cs[i], e * sn[i]);
        }
      }
    }
    store8(dst + lo, a);
    store8(dst + hi, b);
  }
}

template <typename IN, typename OUT>
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<IN, OUT>, p);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "KV append launch");
}

}  // namespace append

int launch_kv_append(const q4_kv_cache& c, int T, const void* k, long long k_stride, const void* v,
                     long long v_stride, int in_dtype, const void* q, long long q_stride, int n_q, void* q_out,
                     const uint64_t* steps, int rot, int interleaved, const int32_t* positions, int32_t* err,
                     const DeviceInfo& dev, cudaStream_t s) {
  append::Params p = {};
  p.kv = kv_tables(c);
  p.k = k, p.v = v, p.q = q;
  p.k_stride = k_stride, p.v_stride = v_stride, p.q_stride = q_stride;
  p.k_cache = c.k, p.v_cache = c.v, p.q_out = q_out;
  p.steps = steps;
  p.positions = positions;
  p.err = err;
  p.T = T, p.D = c.head_dim, p.n_q = n_q, p.rot = rot, p.interleaved = interleaved;
  p.rows = n_q + 2 * c.n_kv;
  // Rows a thread takes: all of a token's while that still fills the device
  // (one set of sines per token and pair), else fewer, down to one.
  const long long want = (long long)dev.sms * 2048;   // resident threads of the device
  const long long per_row = (long long)T * (p.D / append::kChunk);
  int groups = (int)((want + per_row - 1) / per_row);
  if (groups > p.rows) groups = p.rows;
  p.rows_per_group = (p.rows + groups - 1) / groups;
  p.groups = (p.rows + p.rows_per_group - 1) / p.rows_per_group;
  const bool f16 = c.dtype == Q4_F16;
  switch (in_dtype) {
    case Q4_F32:
      return f16 ? append::launch<float, __half>(p, s) : append::launch<float, __nv_bfloat16>(p, s);
    case Q4_F16:
      return f16 ? append::launch<__half, __half>(p, s) : append::launch<__half, __nv_bfloat16>(p, s);
    default:
      return f16 ? append::launch<__nv_bfloat16, __half>(p, s) : append::launch<__nv_bfloat16, __nv_bfloat16>(p, s);
  }
}

}  // namespace q4w
