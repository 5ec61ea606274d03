// Attention of new tokens over a paged cache, the plain form: one warp per
// (token, query head), one key at a time, fp32 throughout.
//
// o = sum_c softmax_c(scale q.k_c) v_c over the cache positions c in
// (P - window, P], c >= 0, P the token's own position; one pass over the keys
// with the running maximum m and sum l of the softmax: a key of score s takes
// m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v.
#include <math_constants.h>

#include "q4w_device.cuh"
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"

namespace q4w {
namespace attn {

constexpr int kThr = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThr) attn_kernel(const __grid_constant__ AttnParams p) {
  pdl_wait();
  constexpr int N = D / 64;   // pairs of elements per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * (kThr / 32) + warp;
  const int tok = (int)(id / p.n_q), h = (int)(id % p.n_q);
  if (tok >= p.T) return;
  int lo = 0, hi = p.kv.n_seqs;   // the first sequence that ends behind tok
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.kv.cu_tokens[mid + 1] <= tok) lo = mid + 1; else hi = mid;
  }
  const int seq = lo;
  if (seq >= p.kv.n_seqs) return;
  if (tok - p.kv.cu_tokens[seq] >= p.max_q) {
    if (p.err && lane == 0) *p.err = 1;
    return;
  }
  const int pos = p.kv.kv_lens[seq] - p.kv.cu_tokens[seq + 1] + tok;
  const int kvh = h / (p.n_q / p.kv.n_kv);
  const T* q = static_cast<const T*>(p.q) + tok * p.q_stride + (long long)h * D;
  float2 qf[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    qf[i] = Half16<T>::unpack(*reinterpret_cast<const uint32_t*>(q + 2 * (lane + 32 * i)));
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -CUDART_INF_F, l = 0.f;
  for (int c = kv_first(pos, p.window); c <= pos; ++c) {
    const int page = kv_page(p.kv, seq, c);
    if (page < 0) {
      if (p.err && lane == 0) *p.err = 1;
      continue;
    }
    const long long row = kv_row(p.kv, page, kvh) + c % p.kv.page_size;
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.k) + row * D);
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.v) + row * D);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 kf = Half16<T>::unpack(kr[lane + 32 * i]);
      s = fmaf(qf[i].x, kf.x, fmaf(qf[i].y, kf.y, s));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float m2 = fmaxf(m, s);
    const float f = m2 == -CUDART_INF_F ? 1.f : expf(m - m2), e = m2 == -CUDART_INF_F ? 0.f : expf(s - m2);
    m = m2;
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 vf = Half16<T>::unpack(vr[lane + 32 * i]);
      o[i].x = fmaf(e, vf.x, o[i].x * f);
      o[i].y = fmaf(e, vf.y, o[i].y * f);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + ((long long)tok * p.n_q + h) * D);
#pragma unroll
  for (int i = 0; i < N; ++i) out[lane + 32 * i] = Half16<T>::pack(o[i].x * inv, o[i].y * inv);
  if (p.lse && lane == 0) p.lse[(long long)tok * p.n_q + h] = l == 0.f ? -CUDART_INF_F : m + logf(l);
}

template <typename T, int D>
static int launch(const AttnParams& p, cudaStream_t s) {
  const long long n = (long long)p.T * p.n_q;
  attn_kernel<T, D><<<(unsigned)((n + kThr / 32 - 1) / (kThr / 32)), kThr, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "attention launch");
}

template <typename T>
static int launch_t(const AttnParams& p, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch<T, 64>(p, s);
    case 128: return launch<T, 128>(p, s);
    case 256: return launch<T, 256>(p, s);
    default: return launch<T, 512>(p, s);
  }
}

}  // namespace attn

size_t attn_ws_bytes(int max_rows, int D, int n_seqs, const DeviceInfo& dev) {
  (void)n_seqs;
  return attn_decode_fits(max_rows, D) ? attn_decode_ws_bytes(max_rows, D, dev) : 0;
}

int launch_kv_attention(const AttnParams& p, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  if (attn_decode_fits(p.max_q * (p.n_q / c.n_kv), c.head_dim)) return launch_attn_decode(p, c, ws, dev, s);
  return c.dtype == Q4_F16 ? attn::launch_t<__half>(p, c.head_dim, s)
                           : attn::launch_t<__nv_bfloat16>(p, c.head_dim, s);
}

}  // namespace q4w
