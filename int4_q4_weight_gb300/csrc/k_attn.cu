// kv_attention: the choice between its kernels, and the joining of split work.
#include "q4w_attn.cuh"
#include "q4w_device.cuh"

namespace q4w {
namespace attn {

// Task: 8 rows (32 when P is 1) of one recorded item and 256 / P of their elements;
// P groups of threads take every P-th part: P = 1, 4 or 16.  Two parts of a tile
// are read by as many threads as there are elements where tiles give tasks enough
// (17 us against 23 with 4 groups), by 4 groups where there are few items (one
// chunk of 64 tokens over 512 keys, with the pass: 16 us against 20).  The 152
// parts of the few rows of a single long sequence are read by 16 groups side by
// side, as there are no other tasks: 16 us with 4 groups, 8 with 16.  Every block
// reads all the records, so the tasks of the few items that were split spread over
// the device whatever CTA recorded them.  (Two blocks on an SM leave a thread 64
// registers, and 108 bytes are spilled.)
constexpr int kJoinThr = 512;

// log2 of P; lg_dv: log2 of the columns.
__device__ __forceinline__ int join_groups(int parts, int used, int lg_dv, bool few) {
  return max(parts <= 4 ? few ? 2 : 0 : parts > 16 && used <= 16 ? 4 : 2, 8 - lg_dv);
}

// Sums of what a thread has of a row, scaled to a running maximum (units of log2 e).
struct JoinSum {
  float4 o;
  float m, l;
  __device__ __forceinline__ void clear() { o = make_float4(0.f, 0.f, 0.f, 0.f), m = -CUDART_INF_F, l = 0.f; }
  __device__ __forceinline__ void add(const float2 ml, const float4 v) {
    const float m2 = fmaxf(m, ml.x), mb = m2 == -CUDART_INF_F ? 0.f : m2;
    const float f0 = ex2(m - mb), f = ex2(ml.x - mb);
    m = m2;
    l = fmaf(ml.y, f, l * f0);
    o.x = fmaf(v.x, f, o.x * f0), o.y = fmaf(v.y, f, o.y * f0), o.z = fmaf(v.z, f, o.z * f0), o.w = fmaf(v.w, f, o.w * f0);
  }
};

template <typename T>
__global__ void __launch_bounds__(kJoinThr, 2) join_kernel(const AttnSplit p, int n_recs, int R, int n_q, int rows, int D, int dv, bool few,
                                                        void* out_, float* lse) {
  __shared__ float4 sum_sh[kJoinThr];
  __shared__ float2 ml_sh[16][8];
  __shared__ int first_sh[kJoinThr + 1];   // tasks before a record's
  __shared__ SplitRec rec_sh[kJoinThr];
  __shared__ int warp_sh[kJoinThr / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg_dv = 31 - __clz(dv);   // 64 to 512
  pdl_wait();
  {
    int n = 0;
    if (threadIdx.x < n_recs) {
      const SplitRec r = p.recs[threadIdx.x];
      rec_sh[threadIdx.x] = r;
      const int g = join_groups(r.last - (int)threadIdx.x / R + 1, r.used, lg_dv, few), lg_rows = g == 0 ? 5 : 3;
      n = r.last < 0 ? 0 : ((r.used + (1 << lg_rows) - 1) >> lg_rows) << (lg_dv + g - 8);
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
    const int lg = join_groups(np, rec.used, lg_dv, few), groups = 1 << lg, lg_cols = lg_dv + lg - 8;
    const int part = threadIdx.x >> (9 - lg), dl = (threadIdx.x >> 3) & ((64 >> lg) - 1);
    const int d = (((sub & ((1 << lg_cols) - 1)) << (6 - lg)) + dl) * 4;
    // row `rr` of the task's first 8: of part 0, and of part i >= 1 at i - 1 steps
    // behind part 1
    const int r0 = (sub >> lg_cols) * (lg == 0 ? 32 : 8) + rr;
    const long long slot0 = (2ll * c0 + 1) * R + lo % R, slot1 = (2ll * c0 + 2) * R + lo % R;
    const float* const o0 = p.part_o + (slot0 * dv + d) * rows + 4 * r0;
    const float* const o1 = p.part_o + (slot1 * dv + d) * rows + 4 * r0;
    const float2* const ml0 = p.part_ml + slot0 * rows + r0;
    const float2* const ml1 = p.part_ml + slot1 * rows + r0;
    const int o_step = 2 * R * dv * rows, ml_step = 2 * R * rows;
    auto part_ml = [&](int i, int row) { return (i == 0 ? ml0 : ml1 + (long long)(i - 1) * ml_step)[row]; };
    auto part_o = [&](int i, int row) {
      return *reinterpret_cast<const float4*>((i == 0 ? o0 : o1 + (long long)(i - 1) * o_step) + 4 * row);
    };
    const uint32_t by_group = 65536u / rec.group + 1;   // rows below 128: row / group = row * this >> 16
    auto write = [&](int lr, const JoinSum& x) {
      const int tok = (int)(lr * by_group >> 16);
      const long long row = (long long)(rec.token + tok) * n_q + rec.head0 + lr - tok * rec.group;
      const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
      *reinterpret_cast<uint2*>(static_cast<T*>(out_) + row * D + rec.col * dv + d) =
          make_uint2(Half16<T>::pack(x.o.x * inv, x.o.y * inv), Half16<T>::pack(x.o.z * inv, x.o.w * inv));
      if (d == 0 && rec.col == 0 && lse) lse[row] = x.l == 0.f ? -CUDART_INF_F : (x.m + log2f(x.l)) * 0.6931471805599453f;
    };
    if (lg == 0) {   // few parts: four rows a thread, their loads side by side
      JoinSum x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k].clear();
#pragma unroll 1
      for (int i = 0; i < np; i += 2) {
        float2 ml[2][4];
        float4 v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool in = i + h < np && r0 + 8 * k < rec.used;
            ml[h][k] = in ? part_ml(i + h, 8 * k) : make_float2(-CUDART_INF_F, 0.f);
            v[h][k] = in ? part_o(i + h, 8 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k].add(ml[h][k], v[h][k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r0 + 8 * k < rec.used) write(r0 + 8 * k, x[k]);
      continue;
    }
    const bool in = r0 < rec.used;
    JoinSum x;
    x.clear();
    if (in) {
      for (int i = part; i < np; i += 4 * groups) {   // four parts at a time
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = i + groups * k;
          ml[k] = at < np ? part_ml(at, 0) : make_float2(-CUDART_INF_F, 0.f);
          v[k] = at < np ? part_o(at, 0) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) x.add(ml[k], v[k]);
      }
    }
    __syncthreads();
    sum_sh[threadIdx.x] = x.o;
    if (dl == 0) ml_sh[part][rr] = make_float2(x.m, x.l);
    __syncthreads();
    if (part == 0 && in) {
      x.clear();
      for (int i = 0; i < groups; ++i) x.add(ml_sh[i][rr], sum_sh[threadIdx.x + (i << (9 - lg))]);
      write(r0, x);
    }
  }
}

}  // namespace attn

int launch_attn_join(const AttnParams& a, const AttnSplit& split, int rows, int D, int dv, bool bf16, int grid, int R,
                     cudaStream_t s) {
  if (grid > attn::kJoinThr) return fail(Q4_ERR_SHAPE, "attention: %d SMs are more than the join handles", grid);
  // items of the call, about: few when their tasks of 32 rows leave most blocks idle
  const long long items = ((long long)a.T * a.n_q / rows + (long long)a.kv.n_seqs * a.kv.n_kv) * (D / dv);
  const bool few = items * 8 <= 2 * grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * grid);
  cfg.blockDim = dim3(attn::kJoinThr);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e =
      bf16 ? cudaLaunchKernelEx(&cfg, attn::join_kernel<__nv_bfloat16>, split, grid, R, a.n_q, rows, D, dv, few, a.out, a.lse)
           : cudaLaunchKernelEx(&cfg, attn::join_kernel<__half>, split, grid, R, a.n_q, rows, D, dv, few, a.out, a.lse);
  return e == cudaSuccess ? Q4_OK : cuda_fail(e, "attention join launch");
}

size_t attn_ws_bytes(long long max_rows, int D, const DeviceInfo& dev) {
  return attn_decode_fits(max_rows, D) ? attn_decode_ws_bytes((int)max_rows, D, dev) : attn_tile_ws_bytes(D, dev);
}

int launch_kv_attention(const AttnParams& p, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  return attn_decode_fits(p.max_q * (p.n_q / c.n_kv), c.head_dim) ? launch_attn_decode(p, c, ws, dev, s)
                                                                  : launch_attn_tile(p, c, ws, dev, s);
}

}  // namespace q4w
