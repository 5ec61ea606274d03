// Attention of few query rows per KV head over a paged cache (decode, and a few
// drafted tokens): rows = new tokens x query heads of the group <= 8 NT.
//
// Mathematics: one pass over the keys with the running maximum and sum of a
// softmax (scores in units of log2 e, so that e^s is one 2^x); the reference is
// moved only when the maximum has grown by 2^8, so that most steps rescale nothing.
// The final division makes the result independent of that choice.
//
// Bound: HBM.  A 16-bit cache element takes part in 8 or 16 multiply-adds, too
// many for the CUDA cores at 6.8 TB/s (3.4e12 elements/s x 8 x 2 is 54 TFLOP/s)
// and too few to fill a 128-row tensor tile, so the keys are the M rows of
// m16n8k16 (no row is padding at 8 query rows) and the query rows its N:
//   S^T[16 keys][8 rows]   = K[16][D] Q^T         (K by ldmatrix as it lies)
//   O^T[D][8 rows]        += V^T[D][16] P^T       (V by transposing ldmatrix)
// P^T is S^T's own registers after a transposition of 8x8 blocks in registers.
// Every warp streams its own units of 16 keys (K, then V) through a private
// ring by 16-byte asynchronous copies, which place the 128-byte swizzle and leave
// zeros for rows that nothing may see, and synchronises with no other warp until
// its CTA's part of the keys is done; 192 KB are in flight on an SM.  (TMA boxes
// of 16 rows moved 17 bytes a cycle and SM at head size 128, where HBM gives 23.)
//
// Split: one CTA per SM.  The steps (one unit per warp) of all (sequence, KV
// head) pairs form one line that is cut into equal shares, so ragged lengths
// and a single long sequence fill the device alike.  A pair that one CTA has
// whole is written out there; else its parts go to the workspace and a second
// kernel, launched ahead (programmatic dependent launch), joins them in the
// order of the keys: the same lengths give the same bits.
//
// Measured with 8 rows a KV head over caches of 1.2 GB: head sizes 64, 128, 256,
// 512 at 6.2, 6.5, 6.5, 6.2 TB/s; one sequence of 131071 keys of 512 in 56 us
// (4.8 TB/s: 10 us are the start, the warps' merge and the join of 152 parts).
#include <math_constants.h>

#include "q4w_attn.cuh"
#include "q4w_device.cuh"
#include "q4w_internal.cuh"

namespace q4w {
namespace dec {

constexpr int kUnit = 16;              // keys per unit
constexpr int kRingBytes = 196608;     // of a CTA

template <int D, int NT>
struct Shape {
  // A warp holds NT D / 4 + NT D / 8 registers of O and Q.  Twelve warps where
  // that leaves them without spills: 8 rows of head size 64 stream at 6.2 TB/s,
  // with eight warps at 5.4; 16 rows of head size 128 at 5.4 (spills), with eight 6.3.
  // Head size 512 takes 255 registers with four warps and spills 32 bytes.
  static constexpr int kWarps = D == 512 ? 4 : NT * D <= 128 ? 12 : 8;
  static constexpr int kSlotBytes = kUnit * D * 2;
  static constexpr int kSlots = kRingBytes / kWarps / kSlotBytes;   // 3, 3, 6, 12: K and V alternate
  static constexpr int kThr = kWarps * 32;
  static constexpr int kStep = kWarps * kUnit;                      // keys per step of the CTA
  static constexpr int kRowPad = D + 4;                             // floats per row of the output staging
  static constexpr int kMergeBytes = kWarps / 2 * NT * 8 * D * 4;    // half the warps' outputs
  static_assert(kMergeBytes >= NT * 8 * kRowPad * 4, "the output staging shares it");
  static_assert(kMergeBytes >= 8 * kRowPad * 4, "the output staging shares it");
  static constexpr size_t kSmem = kRingBytes + kMergeBytes;
};

struct Params {
  AttnParams a;
  AttnSplit split;
  int group;             // query heads per KV head
  int grid;
};

template <int STEP>
__device__ __forceinline__ int steps_of(const Seq& s) {
  return s.n == 0 ? 0 : s.end > s.base ? (s.end - s.base + STEP - 1) / STEP : 1;
}

// ------------------------------------------------------------ instructions ---
// 16 bytes from global to shared memory, zeros where `in` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A walk over the steps of a CTA's share.
template <int STEP>
struct Walk {
  int seq, head, local, n_local;
  Seq s;
  __device__ __forceinline__ void enter(const AttnParams& a) {
    while (seq < a.kv.n_seqs) {
      s = seq_of(a, seq, kUnit);
      n_local = steps_of<STEP>(s);
      if (n_local > 0) return;
      ++seq;
    }
  }
  // One step on; true when a new (sequence, head) begins.
  __device__ __forceinline__ bool next(const AttnParams& a) {
    if (++local < n_local) return false;
    local = 0;
    if (++head == a.kv.n_kv) {
      head = 0;
      ++seq;
      enter(a);
    }
    return true;
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__((Shape<D, NT>::kThr), 1) decode_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, NT>;
  constexpr int W = S::kWarps, SLOTS = S::kSlots, KS = D / 16;
  extern __shared__ __align__(1024) uint8_t ring[];
  float* merge = reinterpret_cast<float*>(ring + kRingBytes);
  __shared__ float2 ml_sh[W][8 * NT];
  __shared__ long long scan_sh[W];
  __shared__ int start_sh[3];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnParams& a = p.a;

  if (threadIdx.x == 0) start_sh[0] = a.kv.n_seqs;
  pdl_wait();
  pdl_trigger();

  // ---- the shares: every thread sums the steps of a run of sequences
  long long total, share;
  {
    const int per = (a.kv.n_seqs + S::kThr - 1) / S::kThr;
    const int q0 = min((int)threadIdx.x * per, a.kv.n_seqs), q1 = min(q0 + per, a.kv.n_seqs);
    long long sum = 0;
    for (int q = q0; q < q1; ++q) sum += (long long)steps_of<S::kStep>(seq_of(a, q, kUnit)) * a.kv.n_kv;
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) scan_sh[warp] = incl;
    __syncthreads();
    total = 0;
    long long before = incl - sum;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += scan_sh[w];
      total += scan_sh[w];
    }
    share = (total + p.grid - 1) / p.grid;
    const long long mine = share * blockIdx.x;
    if (blockIdx.x == 0 && a.err) {
      for (int q = q0; q < q1; ++q)
        if (seq_bad(a, q)) *a.err = 1;
      if (share > 0x7fffffff) *a.err = 1;   // more steps than 32 bits count: hours
    }
    if (threadIdx.x == 0) p.split.recs[blockIdx.x].last = -1;
    if (sum > 0 && mine >= before && mine < before + sum) {
      long long left = mine - before;
      int q = q0, n;
      for (;; ++q) {
        n = steps_of<S::kStep>(seq_of(a, q, kUnit));
        if (left < (long long)n * a.kv.n_kv) break;
        left -= (long long)n * a.kv.n_kv;
      }
      start_sh[0] = q;
      start_sh[1] = (int)(left / n);
      start_sh[2] = (int)(left % n);
    }
    __syncthreads();
  }
  const long long first_step = share * blockIdx.x;
  const int n_steps = (int)max(0ll, min(share, total - first_step));
  if (n_steps == 0 || share > 0x7fffffff) return;

  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring) + warp * SLOTS * S::kSlotBytes;

  Walk<S::kStep> lw;   // of the loads, ahead of the computation
  lw.seq = start_sh[0], lw.head = start_sh[1], lw.local = start_sh[2];
  lw.enter(a);
  Walk<S::kStep> cw = lw;

  // cache rows of the next 32 units of this warp in the walk's sequence, one per
  // lane (-1: a page that is none of the cache, -2: behind the end)
  int l_step = 0, l_half = 0;        // next load: step of the share, 0 = K, 1 = V
  int row_base = -32, rows = -2;
  int l_row = 0;                     // the unit's first row
  int l_slot = 0;                    // its slot
  uint32_t skip = 0;                 // per slot of K: nothing in it counts
  // a lane's 16-byte pieces of a slot: piece c0 (and + 32 for D = 512) of rows
  // r0, r0 + rows at once, ..
  constexpr int PIECES = D / 8, LR = PIECES < 32 ? 32 / PIECES : 1, COPIES = kUnit * PIECES / 32;
  const int r0 = PIECES < 32 ? lane / PIECES : 0, c0 = PIECES < 32 ? lane % PIECES : lane;
  auto issue = [&]() {
    if (l_step < n_steps) {
      const int k0 = lw.s.base + (lw.local * W + warp) * kUnit;
      if (l_half == 0) {
        if (lw.local < row_base || lw.local >= row_base + 32) {
          row_base = lw.local;
          const int pos = lw.s.base + ((row_base + lane) * W + warp) * kUnit;
          rows = -2;
          if (pos < lw.s.end) {
            const int page = kv_page(a.kv, lw.seq, pos);
            rows = page < 0 ? -1 : (int)kv_row(a.kv, page, lw.head) + pos % a.kv.page_size;
            if (page < 0 && a.err) *a.err = 1;
          }
        }
        l_row = __shfl_sync(0xffffffffu, rows, lw.local - row_base);
        skip = l_row < 0 ? skip | (1u << l_slot) : skip & ~(1u << l_slot);
      }
      // rows that a token may see; what lies in the others may be anything, and 0
      // times infinity is no zero
      const int lo = l_row < 0 ? kUnit : kv_first(lw.s.pos0, a.window) - k0, hi = lw.s.end - k0;
      const T* src = static_cast<const T*>(l_half ? a.v : a.k) + (long long)max(l_row, 0) * D + (r0 * D + c0 * 8);
      const uint32_t dst = ring0 + l_slot * S::kSlotBytes;
#pragma unroll
      for (int i = 0; i < COPIES; ++i) {
        const int r = PIECES <= 32 ? r0 + i * LR : i >> 1, c = PIECES <= 32 ? c0 : c0 + 32 * (i & 1);
        copy16(dst + (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (PIECES <= 32 ? i * LR * D : (i >> 1) * D + (i & 1) * 256),
               r >= lo && r < hi);
      }
      l_slot = l_slot + 1 == SLOTS ? 0 : l_slot + 1;
      if (l_half) {
        l_half = 0;
        ++l_step;
        if (l_step < n_steps && lw.next(a)) row_base = -32;
      } else {
        l_half = 1;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");   // an empty one behind the last
  };
  // SLOTS groups are in flight; the oldest has landed, for every lane
  auto landed = [&]() {
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    __syncwarp();
  };
  for (int i = 0; i < SLOTS; ++i) issue();

  // ---- per (sequence, head): the query rows in registers
  uint32_t qf[NT][KS][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  const float sc = a.scale * 1.4426950408889634f;
  auto begin = [&]() {
    const int R = cw.s.n * p.group;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + (lane >> 2);
      const bool in = r < R;
      const int tok = in ? r / p.group : 0;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + (cw.s.cu + tok) * a.q_stride +
                                                            (long long)(cw.head * p.group + r - tok * p.group) * D);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[t][k][0] = in ? q[k * 8 + (lane & 3)] : 0u;
        qf[t][k][1] = in ? q[k * 8 + 4 + (lane & 3)] : 0u;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) m[t][j] = -CUDART_INF_F, l[t][j] = 0.f;
    }
  };
  begin();

  int c_slot = 0;   // next slot to consume
  bool opens = cw.local == 0;
  for (int step = 0; step < n_steps; ++step) {
    // ------------------------------------------------ one unit of 16 keys
    const int k0 = cw.s.base + (cw.local * W + warp) * kUnit;
    const uint32_t ks = ring0 + c_slot * S::kSlotBytes;
    const bool valid = !((skip >> c_slot) & 1);
    c_slot = c_slot + 1 == SLOTS ? 0 : c_slot + 1;
    const uint32_t vs = ring0 + c_slot * S::kSlotBytes;
    c_slot = c_slot + 1 == SLOTS ? 0 : c_slot + 1;
    landed();
    float s[NT][4];
    if (valid) {
      float acc[NT][2][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][h][j] = 0.f;
      const int row = lane & 15;
      const uint32_t rbase = ks + row * 128;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t kf[4];
        ldsm4(rbase + (k >> 2) * 2048 + (((((k & 3) << 1) + (lane >> 4)) ^ (row & 7)) << 4), kf);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma<T>(acc[t][k & 1], kf, qf[t][k][0], qf[t][k][1]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[t][j] = (acc[t][0][j] + acc[t][1][j]) * sc;
    }
    __syncwarp();
    issue();   // into the slot of K
    uint32_t pf[NT][2];
    if (valid) {
      // masks: only units at the ends of what the tokens see
      const int last = cw.s.pos0 + cw.s.n - 1;
      if (k0 + kUnit - 1 > cw.s.pos0 || k0 < kv_first(last, a.window) || k0 + kUnit > cw.s.end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * t + 2 * (lane & 3) + (j & 1), c = k0 + (lane >> 2) + 8 * (j >> 1);
            const int pos = cw.s.pos0 + r / p.group;
            if (c > pos || c < kv_first(pos, a.window) || c >= cw.s.end) s[t][j] = -CUDART_INF_F;
          }
      }
      // the maximum over the 16 keys; the reference moves when it is passed
      bool move = false;
      float mx[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = fmaxf(s[t][j], s[t][j + 2]);
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          mx[t][j] = v;
          move |= v > m[t][j] + Reference<T>::move;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float m2 = fmaxf(m[t][j], mx[t][j] - Reference<T>::below);
            f[j] = m2 == -CUDART_INF_F ? 1.f : ex2(m[t][j] - m2);
            m[t][j] = m2;
            l[t][j] *= f[j];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[t][i][0] *= f[0], o[t][i][1] *= f[1], o[t][i][2] *= f[0], o[t][i][3] *= f[1];
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float m0 = m[t][0] == -CUDART_INF_F ? 0.f : m[t][0], m1 = m[t][1] == -CUDART_INF_F ? 0.f : m[t][1];
        const float e0 = ex2(s[t][0] - m0), e1 = ex2(s[t][1] - m1), e2 = ex2(s[t][2] - m0), e3 = ex2(s[t][3] - m1);
        l[t][0] += e0 + e2;
        l[t][1] += e1 + e3;
        pf[t][0] = transpose8(Half16<T>::pack(e0, e1));
        pf[t][1] = transpose8(Half16<T>::pack(e2, e3));
      }
    }
    landed();
    if (valid) {
      const int row = (lane & 7) + ((lane >> 4) << 3);
      const uint32_t rbase = vs + row * 128;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vf[4];
        ldsm4t(rbase + (i >> 2) * 2048 + (((((i & 3) << 1) + ((lane >> 3) & 1)) ^ (row & 7)) << 4), vf);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma<T>(o[t][i], vf, pf[t][0], pf[t][1]);
      }
    }
    __syncwarp();
    issue();   // into the slot of V

    // ------------------------------------------------ end of this pair's part
    const bool closes = cw.local + 1 == cw.n_local;
    if (!closes && step + 1 < n_steps) {
      ++cw.local;
      continue;
    }
    {
      // the warps' maxima and sums
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = l[t][j];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (lane < 4) ml_sh[warp][8 * t + 2 * lane + j] = make_float2(m[t][j], v);
        }
      __syncthreads();
      const int R = cw.s.n * p.group;
      const bool whole = opens && closes;
      const long long slot = 2ll * blockIdx.x + (opens ? 1 : 0);
      if (opens && !closes && threadIdx.x == 0)   // goes on in the next CTAs
        p.split.recs[blockIdx.x] = {(int)((first_step + step - cw.local + cw.n_local - 1) / share), cw.s.cu, R,
                                    cw.head * p.group, p.group, 0};
      {
        // every warp to the common maximum
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = 8 * t + 2 * (lane & 3) + j;
            float mm = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < W; ++w) mm = fmaxf(mm, ml_sh[w][r].x);
            const float f = m[t][j] == -CUDART_INF_F ? 0.f : ex2(m[t][j] - mm);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[t][i][j] *= f, o[t][i][j + 2] *= f;
          }
        // their sum, pairwise: of n warps the upper n / 2 are added to the first
#pragma unroll
        for (int n = W; n > 1; n -= n / 2) {
          const int half = n / 2;
          if (warp >= n - half && warp < n) {
            float* b = merge + (warp - (n - half)) * NT * 8 * D + lane;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) b[((t * (D / 16) + i) * 4 + j) * 32] = o[t][i][j];
          }
          __syncthreads();
          if (warp < half) {
            const float* b = merge + warp * NT * 8 * D + lane;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][i][j] += b[((t * (D / 16) + i) * 4 + j) * 32];
          }
          __syncthreads();
        }
        if (warp == 0) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                merge[(8 * t + 2 * (lane & 3) + (j & 1)) * S::kRowPad + 16 * i + (lane >> 2) + 8 * (j >> 1)] = o[t][i][j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < NT * 8 * (D / 4); i += S::kThr) {
          const int r = i % (8 * NT), d = 4 * (i / (8 * NT));
          if (r >= R) continue;
          float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) mm = fmaxf(mm, ml_sh[w][r].x);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float2 x = ml_sh[w][r];
            ll += x.x == -CUDART_INF_F ? 0.f : x.y * ex2(x.x - mm);
          }
          const float4 v = *reinterpret_cast<const float4*>(merge + r * S::kRowPad + d);
          if (whole) {
            const int tok = r / p.group;
            const long long row = (long long)(cw.s.cu + tok) * a.n_q + cw.head * p.group + r - tok * p.group;
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + d) =
                make_uint2(Half16<T>::pack(v.x * inv, v.y * inv), Half16<T>::pack(v.z * inv, v.w * inv));
            if (d == 0 && a.lse) a.lse[row] = ll == 0.f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float4*>(p.split.part_o + (slot * D + d) * (8 * NT) + 4 * r) = v;
            if (d == 0) p.split.part_ml[slot * (8 * NT) + r] = make_float2(mm, ll);
          }
        }
        __syncthreads();
      }
    }
    if (step + 1 < n_steps) {
      cw.next(a);
      opens = true;
      begin();
    }
  }
}

template <typename T, int D, int NT>
static int launch(Params& p, const DeviceInfo& dev, cudaStream_t s) {
  using S = Shape<D, NT>;
  static PerDevice attr;
  if (!attr.get(dev.ordinal)) {
    const cudaError_t e = cudaFuncSetAttribute(decode_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)S::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "decode attention smem attribute");
    attr.set(dev.ordinal);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(S::kThr);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_kernel<T, D, NT>, p);
  if (e != cudaSuccess) return cuda_fail(e, "decode attention launch");
  return launch_attn_join(p.a, p.split, 8 * NT, D, D, std::is_same<T, __nv_bfloat16>::value, p.grid, 1, s);
}

// The largest NT.  More rows go to the tiles of 128 rows, although most of a
// tile is padding then: 16 rows of head size 256 took 208 us here and 198 there (64
// sequences of 16384), 32 rows of 128 took 223 and 146 (16 x 8 heads of 8192;
// their O and Q spill here), 32 rows of 64, which do not, 141 and 273.
constexpr int max_nt(int D) { return D >= 256 ? 1 : D == 128 ? 2 : 4; }

template <typename T>
static int launch_t(Params& p, int D, int nt, const DeviceInfo& dev, cudaStream_t s) {
  switch (D) {
    case 64: return nt == 1 ? launch<T, 64, 1>(p, dev, s) : nt == 2 ? launch<T, 64, 2>(p, dev, s) : launch<T, 64, 4>(p, dev, s);
    case 128: return nt == 1 ? launch<T, 128, 1>(p, dev, s) : launch<T, 128, 2>(p, dev, s);
    case 256: return launch<T, 256, 1>(p, dev, s);
    default: return launch<T, 512, 1>(p, dev, s);
  }
}

static int nt_of(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

}  // namespace dec

bool attn_decode_fits(long long max_rows, int D) { return max_rows <= 8 * dec::max_nt(D); }

size_t attn_decode_ws_bytes(int max_rows, int D, const DeviceInfo& dev) {
  return attn_split_bytes(dev.sms, 8 * dec::nt_of(max_rows), D);
}

int launch_attn_decode(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  dec::Params p = {};
  const bool bf16 = c.dtype == Q4_BF16;
  p.a = a;
  p.group = a.n_q / c.n_kv;
  const int nt = dec::nt_of(a.max_q * p.group);
  p.grid = dev.sms;
  p.split = attn_split(ws, p.grid, 8 * nt, c.head_dim);
  return bf16 ? dec::launch_t<__nv_bfloat16>(p, c.head_dim, nt, dev, s)
              : dec::launch_t<__half>(p, c.head_dim, nt, dev, s);
}

}  // namespace q4w
