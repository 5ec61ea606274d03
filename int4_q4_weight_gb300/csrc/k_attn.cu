// kv_attention: the choice between its kernels, and the joining of split work.
#include "q4w_attn.cuh"
#include "q4w_device.cuh"

namespace q4w {
namespace attn {

// Task: 8 rows of one recorded item and 256 / P of their elements; P groups of
// threads take every P-th part (P = 1, 4 or 16: two parts of a tile are read by
// as many threads as there are elements; the 152 parts of the few rows of a
// single long sequence by 16 groups side by side, as there are no other tasks:
// 16 us with 4 groups, 8 with 16; tiles have tasks enough, 17 us against 23).  Every block reads all the
// records, so the tasks of the few items that were split spread over the device
// whatever CTA recorded them.
constexpr int kJoinThr = 512;

__device__ __forceinline__ int join_groups(int parts, int used, int dv) {
  return max(parts <= 4 ? 1 : parts > 16 && used <= 16 ? 16 : 4, 256 / dv);
}

template <typename T>
__global__ void __launch_bounds__(kJoinThr) join_kernel(const AttnSplit p, int n_recs, int R, int n_q, int rows, int D, int dv,
                                                        void* out_, float* lse) {
  __shared__ float4 sum_sh[kJoinThr];
  __shared__ float2 ml_sh[16][8];
  __shared__ int first_sh[kJoinThr + 1];   // tasks before a record's
  __shared__ SplitRec rec_sh[kJoinThr];
  __shared__ int warp_sh[kJoinThr / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  {
    int n = 0;
    if (threadIdx.x < n_recs) {
      const SplitRec r = p.recs[threadIdx.x];
      rec_sh[threadIdx.x] = r;
      n = r.last < 0 ? 0 : (r.used + 7) / 8 * (dv * join_groups(r.last - (int)threadIdx.x / R + 1, r.used, dv) / 256);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) warp_sh[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sh[w];
    first_sh[threadIdx.x + 1] = before + incl;
    if (threadIdx.x == 0) first_sh[0] = 0;
    __syncthreads();
  }
  const int rr = threadIdx.x & 7;   // rows lie side by side in a part
  const int total = first_sh[kJoinThr];
  for (int task = blockIdx.x; task < total; task += gridDim.x) {
    int lo = 0, hi = n_recs;   // the record: the last one that begins at or before the task
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_sh[mid] <= task) lo = mid; else hi = mid;
    }
    const SplitRec rec = rec_sh[lo];
    const int c0 = lo / R, sub = task - first_sh[lo], np = rec.last - c0 + 1;
    const int groups = join_groups(np, rec.used, dv), quads = 64 / groups, col_tasks = dv * groups / 256;
    const int part = (threadIdx.x >> 3) / quads, dl = (threadIdx.x >> 3) % quads, d = (sub % col_tasks * quads + dl) * 4;
    const int lr = sub / col_tasks * 8 + rr;
    const bool in = lr < rec.used;
    auto slot = [&](int i) { return (i == 0 ? 2ll * c0 + 1 : 2ll * (c0 + i)) * R + lo % R; };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, m = -CUDART_INF_F;
    if (in) {
      for (int i = part; i < np; i += 4 * groups) {   // four parts at a time
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = i + groups * k;
          ml[k] = at < np ? p.part_ml[slot(at) * rows + lr] : make_float2(-CUDART_INF_F, 0.f);
          v[k] = at < np ? *reinterpret_cast<const float4*>(p.part_o + (slot(at) * dv + d) * rows + 4 * lr) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float m2 = fmaxf(m, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
        const float mb = m2 == -CUDART_INF_F ? 0.f : m2, f0 = ex2(m - mb);
        m = m2;
        l *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = ex2(ml[k].x - mb);
          l = fmaf(ml[k].y, f, l);
          o.x = fmaf(v[k].x, f, o.x), o.y = fmaf(v[k].y, f, o.y), o.z = fmaf(v[k].z, f, o.z), o.w = fmaf(v[k].w, f, o.w);
        }
      }
    }
    __syncthreads();
    sum_sh[threadIdx.x] = o;
    if (dl == 0) ml_sh[part][rr] = make_float2(m, l);
    __syncthreads();
    if (part == 0 && in) {
      float mm = -CUDART_INF_F;
      for (int i = 0; i < groups; ++i) mm = fmaxf(mm, ml_sh[i][rr].x);
      const float mb = mm == -CUDART_INF_F ? 0.f : mm;
      l = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < groups; ++i) {
        const float f = ex2(ml_sh[i][rr].x - mb);
        const float4 v = sum_sh[threadIdx.x + 8 * quads * i];
        l = fmaf(ml_sh[i][rr].y, f, l);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
      }
      const long long row = (long long)(rec.token + lr / rec.group) * n_q + rec.head0 + lr % rec.group;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(static_cast<T*>(out_) + row * D + rec.col * dv + d) =
          make_uint2(Half16<T>::pack(o.x * inv, o.y * inv), Half16<T>::pack(o.z * inv, o.w * inv));
      if (d == 0 && rec.col == 0 && lse) lse[row] = l == 0.f ? -CUDART_INF_F : (mm + log2f(l)) * 0.6931471805599453f;
    }
  }
}

}  // namespace attn

int launch_attn_join(const AttnParams& a, const AttnSplit& split, int rows, int D, int dv, bool bf16, int grid, int R,
                     cudaStream_t s) {
  if (grid > attn::kJoinThr) return fail(Q4_ERR_SHAPE, "attention: %d SMs are more than the join handles", grid);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * grid);
  cfg.blockDim = dim3(attn::kJoinThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e =
      bf16 ? cudaLaunchKernelEx(&cfg, attn::join_kernel<__nv_bfloat16>, split, grid, R, a.n_q, rows, D, dv, a.out, a.lse)
           : cudaLaunchKernelEx(&cfg, attn::join_kernel<__half>, split, grid, R, a.n_q, rows, D, dv, a.out, a.lse);
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
