// Attention of many query rows per KV head over an int8 paged cache: the queries as fp16,
// what the kernel of q4w_attn_tile.cuh is instantiated for, and its launch.
#include "q4w_attn_tile.cuh"

namespace q4w {
namespace tile {

// bf16 queries as fp16, a row times query_factor().  A warp a row; HBM, of a few per cent of the
// attention's time.
constexpr int kQueryThr = 256;
template <int D>
__global__ void __launch_bounds__(kQueryThr) query_kernel(const __nv_bfloat16* q, long long stride, int T, int n_q, __half* out, float* row_scale) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = D / 64;   // pairs of elements a lane
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kQueryThr / 32) + (threadIdx.x >> 5);
  if (row >= (long long)T * n_q) return;
  const long long tok = row / n_q;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(q + tok * stride + (row - tok * n_q) * D) + lane * E;
  uint32_t x[E];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(x[i]) : "l"(src + i) : "memory");   // behind the wait
    const float2 f = Half16<__nv_bfloat16>::unpack(x[i]);
    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  const float f = query_factor(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * D) + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float2 v = Half16<__nv_bfloat16>::unpack(x[i]);
    dst[i] = Half16<__half>::pack(v.x * f, v.y * f);
  }
  if (lane == 0) row_scale[row] = 1.f / f;
}

static int launch_queries(const AttnParams& a, int D, __half* out, float* row_scale, cudaStream_t s) {
  const long long rows = (long long)a.T * a.n_q;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + kQueryThr / 32 - 1) / (kQueryThr / 32)));
  cfg.blockDim = dim3(kQueryThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const auto* q = static_cast<const __nv_bfloat16*>(a.q);
  const cudaError_t e = D == 64    ? cudaLaunchKernelEx(&cfg, query_kernel<64>, q, a.q_stride, a.T, a.n_q, out, row_scale)
                        : D == 128 ? cudaLaunchKernelEx(&cfg, query_kernel<128>, q, a.q_stride, a.T, a.n_q, out, row_scale)
                        : D == 256 ? cudaLaunchKernelEx(&cfg, query_kernel<256>, q, a.q_stride, a.T, a.n_q, out, row_scale)
                                   : cudaLaunchKernelEx(&cfg, query_kernel<512>, q, a.q_stride, a.T, a.n_q, out, row_scale);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "attention queries launch");
}

template <typename T>
static int launch_t(Params& p, int D, const DeviceInfo& dev, cudaStream_t s) {
  switch (D) {
    case 64: return launch<T, 64, true>(p, dev, s);
    case 128: return launch<T, 128, true>(p, dev, s);
    case 256: return launch<T, 256, true>(p, dev, s);
    default: return launch<T, 512, true>(p, dev, s);
  }
}

}  // namespace tile

// The parts, then T tokens' rows of bf16 queries as fp16 and their factors (0 tokens: fp16 queries).
size_t attn_tile_q8_ws_bytes(long long T, int n_q, int D, const DeviceInfo& dev) {
  return attn_tile_ws_bytes(D, dev) + attn_up256((size_t)T * n_q * D * 2) + attn_up256((size_t)T * n_q * 4);
}

int launch_attn_tile_q8(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  tile::Params p = {};
  const bool bf16 = c.dtype == Q4_BF16;
  const int D = c.head_dim;
  p.box = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : 16;
  p.group = a.n_q / c.n_kv;
  p.tokens = tile::kRows / p.group;
  p.a = a;
  if (bf16) {
    char* at = static_cast<char*>(ws) + attn_tile_ws_bytes(D, dev);
    __half* q16 = reinterpret_cast<__half*>(at);
    float* row_scale = reinterpret_cast<float*>(at + attn_up256((size_t)a.T * a.n_q * D * 2));
    const int st = tile::launch_queries(a, D, q16, row_scale, s);
    if (st != Q4_OK) return st;
    p.a.q = q16;
    p.a.q_stride = (long long)a.n_q * D;
    p.row_scale = row_scale;
  }
  const int st = encode_query_rows(&p.tm_q, p.a.q, false, D, a.n_q, a.T, p.a.q_stride, p.group, p.tokens);
  if (st != Q4_OK) return st;
  p.pairs = dev.sms / 2;
  p.wait_limit = wait_limit();
  p.dev_err = device_error_word();
  p.split = attn_split(ws, dev.sms, tile::kRows, D < 256 ? D : 256);
  return bf16 ? tile::launch_t<__nv_bfloat16>(p, D, dev, s) : tile::launch_t<__half>(p, D, dev, s);
}

}  // namespace q4w
