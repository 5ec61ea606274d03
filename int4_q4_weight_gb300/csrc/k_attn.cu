// kv_attention: the choice between its kernels, and the joining of split work.
#include "q4w_attn.cuh"
#include "q4w_device.cuh"

namespace q4w {
namespace attn {

// Block: 64 elements of 8 rows of one item at a time; four groups of threads
// take every fourth part.  The blocks of an item take its row groups in turn.
constexpr int kJoinThr = 512;

template <typename T>
__global__ void __launch_bounds__(kJoinThr) join_kernel(const __grid_constant__ AttnParams a, const AttnSplit p,
                                                        int group, int rows, int D, int dv, int align) {
  __shared__ float4 sum_sh[kJoinThr];
  __shared__ float l_sh[4][8];
  pdl_wait();
  const int c0 = blockIdx.x;
  const SplitRec rec = p.recs[c0];
  if (rec.last < 0) return;
  const Seq s = seq_of(a, rec.seq, align);
  const int cols = D / dv, tile = rec.tile / cols, tokens = rows / group;   // a tile has whole tokens
  const int used = min(tokens, s.n - tile * tokens) * group;                // its rows
  const int part = threadIdx.x >> 7, rr = (threadIdx.x >> 4) & 7, d = blockIdx.y * 64 + 4 * (threadIdx.x & 15);
  const int np = rec.last - c0 + 1;
  for (int r0 = blockIdx.z * 8; r0 < used; r0 += gridDim.z * 8) {
    const int lr = r0 + rr;
    const bool in = lr < used;
    auto slot = [&](int i) { return (i == 0 ? 2ll * c0 + 1 : 2ll * (c0 + i)) * rows + lr; };
    float mm = -CUDART_INF_F;
    if (in) {
      for (int i = threadIdx.x & 15; i < np; i += 16) mm = fmaxf(mm, p.part_ml[slot(i)].x);
    }
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (in) {
#pragma unroll 4
      for (int i = part; i < np; i += 4) {
        const float2 ml = p.part_ml[slot(i)];
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(i) * dv + d);
        const float f = ml.x == -CUDART_INF_F ? 0.f : ex2(ml.x - mm);
        l = fmaf(ml.y, f, l);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
      }
    }
    __syncthreads();
    sum_sh[threadIdx.x] = o;
    if ((threadIdx.x & 15) == 0) l_sh[part][rr] = l;
    __syncthreads();
    if (part == 0 && in) {
      l = (l_sh[0][rr] + l_sh[1][rr]) + (l_sh[2][rr] + l_sh[3][rr]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const float4 v = sum_sh[threadIdx.x + 128 * i];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      const int tok = tile * tokens + lr / group, col = rec.tile % cols;
      const long long row = (long long)(s.cu + tok) * a.n_q + rec.head * group + lr % group;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + col * dv + d) =
          make_uint2(Half16<T>::pack(o.x * inv, o.y * inv), Half16<T>::pack(o.z * inv, o.w * inv));
      if (d == 0 && col == 0 && a.lse) a.lse[row] = l == 0.f ? -CUDART_INF_F : (mm + log2f(l)) * 0.6931471805599453f;
    }
  }
}

}  // namespace attn

int launch_attn_join(const AttnParams& a, const AttnSplit& split, int group, int rows, int D, int dv, int align,
                     bool bf16, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, dv / 64, rows / 8 < 4 ? rows / 8 : 4);
  cfg.blockDim = dim3(attn::kJoinThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e =
      bf16 ? cudaLaunchKernelEx(&cfg, attn::join_kernel<__nv_bfloat16>, a, split, group, rows, D, dv, align)
           : cudaLaunchKernelEx(&cfg, attn::join_kernel<__half>, a, split, group, rows, D, dv, align);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "attention join launch");
}

size_t attn_ws_bytes(int max_rows, int D, int n_seqs, const DeviceInfo& dev) {
  (void)n_seqs;
  return attn_decode_fits(max_rows, D) ? attn_decode_ws_bytes(max_rows, D, dev) : attn_tile_ws_bytes(D, dev);
}

int launch_kv_attention(const AttnParams& p, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  return attn_decode_fits(p.max_q * (p.n_q / c.n_kv), c.head_dim) ? launch_attn_decode(p, c, ws, dev, s)
                                                                  : launch_attn_tile(p, c, ws, dev, s);
}

}  // namespace q4w
