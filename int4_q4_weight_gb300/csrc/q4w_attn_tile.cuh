// Attention of many query rows per KV head over a paged cache (prefill chunks,
// prompts): tiles of 128 query rows on the 5th-generation tensor cores.  The kernel,
// for a 16-bit cache and for one of int8 codes; k_attn_tile*.cu instantiate it.
//
// A tile's rows are (token, query head of the group) pairs, so all heads of a
// group share the keys that are read.  One pass over the keys, 128 a step:
//   S[128 rows][128 keys] = Q K^T     A = Q, B = K, both in shared memory
//   P = 2^(S scale log2(e) - m)       two threads per row, half of the keys
//                                     each, S read from TMEM, P (16 bits)
//                                     written over it
//   O[128 rows][DV]      += P V       A = P in TMEM, B = V in shared memory
// with the running reference m and sum of each row in its threads.  m is moved
// only when the maximum has grown by 2^8, so O (in TMEM) is rarely rescaled.
// Two S tiles alternate: the scores of step j + 1 are formed while the softmax
// of step j runs.  TMEM: S 2 x 128 columns, O 256 = all 512.  Head size 512 does
// not fit: its two column halves of O are items of their own, which form the
// scores twice (1.5 times the products).
//
// Two CTAs, a cluster, take the two tiles of a pair as one (cta_group::2): an MMA
// of 256 rows takes Q, P and the accumulators of each CTA's 128 rows from that
// CTA, and half of the keys of K (of the columns of V) from each.  Alone, a CTA
// is bound by its shared memory at head size 256: a step's products read 128 KB
// for QK^T and 64 KB for PV, and 128 KB of K and V are written, 2560 cycles at 128
// bytes a cycle against 2048 of products, and 3450 were measured, also when the
// two CTAs shared their loads by multicast.  As a pair it is 96, 32 and 64 KB, and
// the rings hold two and a half steps.
//
// Warps: 0-7 softmax (warp w the rows 32 (w mod 4) .., keys 64 (w div 4) ..), 8
// issues the MMAs in the even CTA, and in the odd one passes on to it that slots
// have landed, 9 and 10 the loads of K and of V, 11 those of the next item's
// query rows (a box of whole tokens: a tile has floor(128 / group) of them).
// The softmax is written to be short: a path that is taken once per item and
// unrolled to hundreds of instructions cost 20000 cycles of instruction fetches.
// K and V have a ring of slots each, so that the next keys load while the values
// wait for P: K slots of [64 keys][<= 256 dims], V slots of [128 keys][<= 128
// columns], loaded in boxes of 16 to 64 rows (the page size's share), 128-byte
// swizzle.  A slot is as large as the ring allows: waiting for one and releasing
// it costs the issuing thread about 100 cycles.
//
// Split: the steps of all items (sequence, KV head, tile) form one line that is
// cut into equal shares, one CTA per SM; causal tiles of any length and ragged
// sequences balance, and a short chunk over a long cache is split along the
// keys.  Parts are joined by a second kernel in the order of the keys.
//
// Measured: four ragged prompts of up to 4096 tokens over contexts of up to 8192
// (8 query heads on 1 KV head of 256, 326 GFLOP): 215 us with the join from a graph,
// 1.5 PFLOP/s, and 228 us a call from Python, 1.43; the tensor pipe active for 79 % of
// the cycles of the busy SMs.  A step takes 2350 cycles; what else is lost lies at the
// ends of items, where O is read out before the next item may write it, and in the
// join.  The same prompts with other heads, from a graph: 8 on 1 of 512 (653 GFLOP,
// the scores formed twice) 585 us, 1.12 PFLOP/s; 16 on 2 of 128
// (326 GFLOP) 336 us, 0.97; 32 on 4 of 64, where half of the second product is zeros,
// 581 us, 0.56.
//
// The int8 cache.  K and V are widened on the way: instead of the two warps that issue
// TMA loads, eight warps for K and six for V read codes and scales (a slot ahead, in
// registers), and write fp16 tiles in the same swizzled layout.
//   K: code * scale has 19 significant bits, so it is held as two fp16 numbers, whose
//      sum is exact down to fp16's subnormal step, and the scores are two products:
//      one alone would put 3e-4 on a score, and on the log-sum of a row of few keys.
//   V: code * scale rounded once to fp16.  P is fp16 too, in two pieces for fp16 queries.
// Queries are fp16: those in bf16 are converted first (k_attn_tile_q8.cu) with a power of
// two for each row, which its softmax threads take into the scale.  The products are 1.5
// times those of a 16-bit cache (twice with two pieces of P).
//
// Bound: the latency of the roles, which share four schedulers.  Four prompts of up to
// 2048 tokens over up to 8192 keys (8 heads on 1 of 256, 181 GFLOP of a 16-bit cache's products), bf16:
// 211 us with queries and join, 16-bit cache 124; fp16, with a product more, 234.  A step takes 4200
// cycles, three quarters of them products.  What brought it there from 330: three warps each for K and V could not widen a step
// in its time (an instruction of theirs takes 12 cycles), so fourteen; a table lookup and
// walk per step for all of them in one warp (a ring of plans); reads for the next slot behind all
// the stores (between them they share the scoreboards that the stores wait by); the issuing
// thread's instructions between two products (each waits its turn with five warps): one lane, one
// barrier for both pieces of K, no relay through the other CTA.  Roles of a scheduler share their
// code, as the instruction cache does not hold all of it: K and V on the same schedulers cost
// 20 us.  Slots of half the size, or the softmax 16 scores at a time, were slower.
#pragma once

#include <cuda.h>

#include "q4w_attn.cuh"
#include "q4w_codes.cuh"
#include "q4w_device.cuh"
#include "q4w_tc_pair.cuh"

namespace q4w {
namespace tile {

constexpr int kRows = 128, kKeys = kv_tile_keys;
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps, kKWarp = kMmaWarp + 1, kVWarp = kKWarp + 1, kQWarp = kVWarp + 1;
// The int8 cache: warps 10 and 11 issue and load the queries, eight widen K and six V (two pieces of K
// take half as many instructions again).  24 warps have 80 registers each, so the softmax
// holds 32 scores at a time and reads them twice.
constexpr int kWidenK = 8, kWidenV = 6;
constexpr int kThr = (kQWarp + 1) * 32, kThrQ8 = (kKWarp + 1 + kWidenK + kWidenV) * 32;
constexpr long long kDrainCycles = 2000000000LL;
constexpr long long kShortDrainCycles = 4000000LL;   // aborting: copies in flight land well within this
constexpr int kBadRing = 16;

template <int D, bool Q8 = false>
struct Shape {
  static constexpr int kDV = D < 256 ? D : 256;              // columns of O of an item
  static constexpr int kParts = D / kDV;                     // items per tile
  static constexpr int kN = D == 64 ? 128 : kDV;             // columns of the MMA (D = 64: the odd CTA's are zeros)
  static constexpr int kKD = D < 256 ? D : 256;   // dims of a K slot
  static constexpr int kNK = (Q8 ? 2 : 1) * (D / kKD);       // K slots per step (int8 cache: upper and lower pieces)
  static constexpr int kKSlot = kKeys / 2 * kKD * 2;         // bytes: 8, 16, 32, 32 KB
  static constexpr int kVSlot = kKeys * kN;                  // all keys of a step, kN / 2 columns a CTA: 16, 16, 32, 32 KB
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKSlots = D <= 128 ? 6 : Q8 && D == 256 ? 3 : 2;   // rings of K and of V
  static constexpr int kVSlots = D <= 128 ? 6 : D == 256 ? (Q8 ? 2 : 3) : 1;
  static constexpr int kThreads = Q8 ? kThrQ8 : kThr;
  static constexpr int kRing = kKSlots * kKSlot + kVSlots * kVSlot;
  static_assert(kQBytes + kRing <= 229376, "shared memory");
  static constexpr size_t kSmem = kQBytes + kRing;   // with the static part, all 227 KB
};

struct Params {
  CUtensorMap tm_k, tm_v, tm_q;
  AttnParams a;
  AttnSplit split;
  unsigned* dev_err;
  long long wait_limit;
  int group, tokens;     // query heads per KV head, tokens of a tile (a pair has twice as many)
  int total_rows, pairs; // pairs: of CTAs
  int box;               // rows of a TMA box: 16, 32 or 64, a divisor of the page size
  const float* row_scale;   // int8 cache, bf16 queries: what the rows [T][n_q] were divided by, else NULL
};

// Keys that pair t of tiles of a sequence sees, and its steps; `tokens`: of a pair.
__device__ __forceinline__ KvSpan span_of(const AttnParams& a, const Seq& s, int tokens, int t, int box) {
  return kv_span(s.pos0, s.n, s.end, a.window, tokens, t, box);
}
__device__ __forceinline__ int tiles_of(const Seq& s, int tokens) { return (s.n + tokens - 1) / tokens; }

// A walk over the items of a CTA's share: for each sequence its heads, their
// column parts, their tiles.
struct Walk {
  int seq, head, part, t, n_tiles;
  int local;             // step of the item
  Seq s;
  KvSpan x;
};
template <int PARTS>
__device__ __forceinline__ void walk_item(Walk& w, const Params& p) { w.x = span_of(p.a, w.s, 2 * p.tokens, w.t, p.box); }
// To the next item (the caller knows that there is one).
template <int PARTS>
__device__ __forceinline__ void walk_next(Walk& w, const Params& p) {
  w.local = 0;
  if (++w.t == w.n_tiles) {
    w.t = 0;
    if (++w.part == PARTS) {
      w.part = 0;
      if (++w.head == p.a.kv.n_kv) {
        w.head = 0;
        do {
          ++w.seq;
          if (w.seq >= p.a.kv.n_seqs) return;
          w.s = seq_of(p.a, w.seq, p.box);
          w.n_tiles = tiles_of(w.s, 2 * p.tokens);
        } while (w.n_tiles == 0);
      }
    }
  }
  walk_item<PARTS>(w, p);
}

// The int8 cache's kernel has five roles whose loops do not fit the instruction cache side by side
// when every wait is expanded: there what follows the first look is a function.
static __device__ __noinline__ bool wait_call(uint32_t bar, uint32_t parity, long long limit, volatile int* abort_flag, unsigned* err) {
  return tc::mbar_wait(bar, parity, limit, abort_flag, err);
}
template <bool CALL>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, long long limit, volatile int* abort_flag, unsigned* err) {
  if constexpr (CALL) return tc::mbar_probe(bar, parity) || wait_call(bar, parity, limit, abort_flag, err);
  else return tc::mbar_wait(bar, parity, limit, abort_flag, err);
}

// Instruction descriptor, kind::f16: fp32 accumulators, A and B of one 16-bit
// type, M = 256 (both CTAs' rows), N = n; bit 16: B is MN-major (its N index is the contiguous one).
__host__ __device__ constexpr uint32_t idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(2 * kRows >> 4) << 24);
}
// Descriptors as their low words: the high word is a constant of the layout, and a step along an
// operand adds to the low word alone (addresses are below 2^18).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t id, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %5, 0;\n mov.b64 da, {%1, %3};\n mov.b64 db, {%2, %3};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(id), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t id, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(id), "r"(accum)
      : "memory");
}
// MN-major operand in the 128-byte swizzle: 64 elements of MN are one 128-byte
// row per K index, eight K rows (1024 bytes) a group (stride byte offset), the
// next 64 elements of MN `lbo` bytes further (leading byte offset).
__device__ __host__ __forceinline__ constexpr uint64_t desc_mn_sw128(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// ------------------------------------------------- widening an int8 cache ---
// What is needed of a step to read its keys; one warp writes it for all.
constexpr int kPlans = 4;   // steps ahead
struct Plan {
  int row[8];             // the cache row where box b of the step begins, -1: nothing to read
  int k0, lo, end, part;  // the step's first key, the keys that the tile sees, the part of the columns
};
struct StepRows {
  int row;                // lane b (mod 8): of box b
  int k0, lo, end;
};
// A warp's share of one slot: ROWS keys from key `key0` of the step on, LPR 16-byte pieces of
// codes each, from element `dim` of the head (of D) on.  Lanes take pieces of 32 / LPR keys at once;
// warp w every WARPS-th such group.  All its groups are in registers: a group is read for the
// next slot as soon as it is written to this one, so that a slot's time covers the read.
template <int ROWS, int LPR, int WARPS, int D>
struct Widen {
  static constexpr int kAtOnce = 32 / LPR, kAll = ROWS / kAtOnce, kGroups = (kAll + WARPS - 1) / WARPS, kApart = WARPS * kAtOnce;
  static_assert(kApart % 8 == 0, "a lane's keys share their place in the swizzle");
  uint4 code[kGroups];
  __half scale[kGroups];
  uint32_t none = 0;   // bit u: the group's row of this lane counts as zeros

  static __device__ __forceinline__ int piece(int lane) { return lane % LPR; }
  static __device__ __forceinline__ bool here(int w, int u) { return w + WARPS * u < kAll; }   // the same for the whole warp

  // ZERO: keys that no row sees are zeros (V; of K they are masked, and any code is a number).
  // codes, scales: of this lane's piece of row 0 of the cache.
  template <bool ZERO>
  __device__ __forceinline__ void load(const int8_t* codes, const __half* scales, const StepRows& st, int lg_box, int key0, int w, int u, int lane) {
    if (!here(w, u)) return;
    const int k = key0 + w * kAtOnce + lane / LPR + u * kApart, from = __shfl_sync(0xffffffffu, st.row, k >> lg_box), pos = st.k0 + k;
    const bool in = from >= 0 && (!ZERO || (pos >= st.lo && pos < st.end));
    const int row = in ? from + (k & ((1 << lg_box) - 1)) : 0;
    code[u] = *reinterpret_cast<const uint4*>(codes + (long long)row * D);
    scale[u] = scales[(long long)row * (D / 32)];
    none = in ? none & ~(1u << u) : none | 1u << u;
  }
  // Into the slot(s): rows of 128 bytes, 64 elements, ROWS rows a slab, 128-byte swizzle.  TWO:
  // the rest that the rounding to fp16 leaves goes to `second`.  Neighbouring lanes of every
  // other slab write their second piece first: all banks at once.
  static __device__ __forceinline__ uint32_t place(int w, int lane, int piece) {
    const int r = w * kAtOnce + lane / LPR, c = lane % LPR, odd = (c >> 2) & 1;
    return (c >> 2) * (ROWS * 128) + r * 128 + (((2 * (c & 3) + (piece ^ odd)) ^ (r & 7)) << 4);
  }
  template <bool TWO>
  __device__ __forceinline__ void store(uint32_t first, uint32_t second, uint32_t p0, uint32_t p1, int w, int u, int lane) const {
    if (!here(w, u)) return;
    const bool odd = (lane % LPR) & 4;
    const __half2 s = __half2half2((none >> u) & 1 ? __ushort_as_half(0) : scale[u]);
    const uint4 x = code[u];
    const uint32_t word[4] = {(odd ? x.z : x.x) ^ 0x80808080u, (odd ? x.w : x.y) ^ 0x80808080u, (odd ? x.x : x.z) ^ 0x80808080u,
                              (odd ? x.y : x.w) ^ 0x80808080u};
    uint32_t hi[8], rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t n = i & 1 ? two_codes<2, 3>(word[i >> 1]) : two_codes<0, 1>(word[i >> 1]);
      const __half2 v = *reinterpret_cast<const __half2*>(&n), h = __hmul2(v, s);
      hi[i] = *reinterpret_cast<const uint32_t*>(&h);
      if constexpr (TWO) {
        const __half2 l = __hfma2(v, s, __hneg2(h));
        rest[i] = *reinterpret_cast<const uint32_t*>(&l);
      }
    }
    auto put = [&](uint32_t base, const uint32_t (&v)[8]) {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(base + p0), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(base + p1), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    };
    put(first + u * (kApart * 128), hi);
    if constexpr (TWO) put(second + u * (kApart * 128), rest);
  }
};

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__((Shape<D, Q8>::kThreads), 1) tile_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, Q8>;
  using P16 = typename std::conditional<Q8, __half, T>::type;   // of the operands
  // P as two fp16 pieces where the output is fp16 too, as in the kernel for few rows: V is rounded,
  // and with one piece the roundings' sum would be 1.6 times that of the output alone
  constexpr bool SPLIT_P = Q8 && std::is_same<T, __half>::value;
  constexpr int NKS = S::kKSlots, NVS = S::kVSlots, NS = NKS + NVS, PARTS = S::kParts, kThr = S::kThreads;
  constexpr bool BF16 = std::is_same<P16, __nv_bfloat16>::value;
  constexpr int kIssueWarp = Q8 ? kMmaWarp + 2 : kMmaWarp, kQueryWarp = Q8 ? kIssueWarp + 1 : kQWarp;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if (tc::smem_u32(smem) & 1023) {   // the swizzle needs it; there is no room to move the buffers
    pdl_wait();
    if (threadIdx.x == 0) {
      p.split.recs[blockIdx.x].last = -1;   // the join reads every CTA's record
      atomicOr(p.dev_err, 1u);
    }
    return;
  }
  uint8_t* ring = smem + S::kQBytes;
  __shared__ uint64_t bars[2 * NS + 7];
  __shared__ uint64_t plan_bars[Q8 ? 2 * kPlans : 1];   // an entry is written; it has been read
  __shared__ Plan plans[Q8 ? kPlans : 1];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ int start_sh[3];
  __shared__ long long left_sh;
  __shared__ long long scan_sh[kThr / 32];
  __shared__ uint32_t bad_sh[kBadRing];   // per step: boxes whose page is none of the cache
  __shared__ float row_sh[2][2][kRows];   // per half of the keys: the rows' maxima of a step, their sums of an item
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, rank = blockIdx.x & 1;   // clusters of two along x
  const AttnParams& a = p.a;
  const uint32_t full0 = tc::smem_u32(bars), empty0 = full0 + 8 * NS;
  const uint32_t qfull = empty0 + 8 * NS, qempty = qfull + 8, sfull0 = qempty + 8, pready0 = sfull0 + 16,
                 drain = pready0 + 16;
  volatile int* abort_flag = &abort_sh;

  if (warp == 0) {
    if (lane == 0) abort_sh = 0, start_sh[0] = -1;
    if (lane < 2 * NS + 7) {
      unsigned count = 1;
      // the even CTA's barriers for what its MMAs wait for count both CTAs
      if (rank == 0 && (lane < NS || lane == 2 * NS)) count = 2;                                 // full, qfull
      if (Q8 && rank == 0 && lane < NS) count = 2 * (lane < NKS ? kWidenK : kWidenV);
      if (lane == 2 * NS + 4 || lane == 2 * NS + 5) count = rank == 0 ? 2 * kSoftWarps : 1;      // pready
      tc::mbar_init(tc::smem_u32(bars + lane), count);
    }
    tc::mbar_fence_init();
  }
  if (Q8 && warp == 1) {
    if (lane < 2 * kPlans) tc::mbar_init(tc::smem_u32(plan_bars + lane), lane < kPlans ? 1 : kWidenK + (D == 64 && rank == 1 ? 0 : kWidenV));
    tc::mbar_fence_init();
  }
  if (warp == kIssueWarp) tc::tmem_alloc_pair(tc::smem_u32(&tmem_sh), 512);
  if (lane == 0 && (warp == kQueryWarp || (!Q8 && (warp == kKWarp || warp == kVWarp)))) {
    const CUtensorMap* m = warp == kQueryWarp ? &p.tm_q : warp == kKWarp ? &p.tm_k : &p.tm_v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  pdl_wait();
  pdl_trigger();

  // ---- the shares: a warp per sequence, a lane per tile; the sums in the ring,
  // which holds nothing yet
  long long total, share;
  {
    long long* steps_sh = reinterpret_cast<long long*>(ring);   // steps of one head and part of each sequence
    static_assert(S::kRing >= kMaxSeqs * 8, "the sums fit the ring");
    for (int q = warp; q < a.kv.n_seqs; q += kThr / 32) {
      const Seq s = seq_of(a, q, p.box);
      long long sum = kv_tile_steps(s.pos0, s.n, s.end, a.window, 2 * p.tokens, p.box, lane, 32);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        steps_sh[q] = sum;
        if (blockIdx.x == 0 && a.err && seq_bad(a, q)) *a.err = 1;
      }
    }
    __syncthreads();
    const int per = (a.kv.n_seqs + kThr - 1) / kThr;
    const int q0 = min((int)threadIdx.x * per, a.kv.n_seqs), q1 = min(q0 + per, a.kv.n_seqs);
    const long long times = (long long)a.kv.n_kv * PARTS;
    long long sum = 0;
    for (int q = q0; q < q1; ++q) sum += steps_sh[q] * times;
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
    for (int w = 0; w < kThr / 32; ++w) {
      if (w < warp) before += scan_sh[w];
      total += scan_sh[w];
    }
    share = (total + p.pairs - 1) / p.pairs;
    const long long mine = share * pair;
    if (sum > 0 && mine >= before && mine < before + sum) {
      long long left = mine - before;
      int q = q0;
      while (left >= steps_sh[q] * times) left -= steps_sh[q++] * times;
      const int hp = (int)(left / steps_sh[q]);
      start_sh[0] = q;
      start_sh[1] = hp / PARTS;
      start_sh[2] = hp % PARTS;
      left_sh = left % steps_sh[q];
    }
    if (threadIdx.x == 0) p.split.recs[blockIdx.x].last = -1;
    tc::fence_proxy_async();   // the sums' last use, before the ring's first loads
    __syncthreads();
  }
  const long long first_step = share * pair;
  int n_steps = start_sh[0] < 0 ? 0 : kv_share_steps(total, share, first_step);
  if (n_steps < 0) {   // more steps than 32 bits count: hours
    if (threadIdx.x == 0 && a.err) *a.err = 1;
    n_steps = 0;
  }
  Walk w = {};
  if (n_steps > 0) {
    // the tile: every warp scans the sequence's tiles, 32 at a time
    w.seq = start_sh[0], w.head = start_sh[1], w.part = start_sh[2];
    w.s = seq_of(a, w.seq, p.box);
    w.n_tiles = tiles_of(w.s, 2 * p.tokens);
    long long left = left_sh;
    for (int t0 = 0;; t0 += 32) {
      const int n = t0 + lane < w.n_tiles ? span_of(a, w.s, 2 * p.tokens, t0 + lane, p.box).steps : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > left);
      if (past) {
        const int at = __ffs(past) - 1;
        w.t = t0 + at;
        w.local = (int)left - __shfl_sync(0xffffffffu, incl - n, at);
        break;
      }
      left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    walk_item<PARTS>(w, p);
  }
  tc::fence_before();
  // both CTAs' barriers are initialised, and TMEM allocated, before either signals
  // the other
  tc::cluster_arrive_release();
  tc::cluster_wait();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_sh;
  const uint32_t q_addr = tc::smem_u32(smem), ring0 = tc::smem_u32(ring);
  const uint32_t v_ring0 = ring0 + NKS * S::kKSlot;
  const uint32_t o_tmem = tmem + 256;

  // A step's boxes, lane b the box b: the block-table entry is fetched a step
  // before it is needed (the load takes longer than a slot's products).
  struct Boxes {
    int entry, off, head, part;   // entry -2: nothing to load
  };
  auto fetch = [&](const Walk& y) {
    Boxes x = {-2, 0, y.head, y.part};
    const int pos = y.x.base + y.local * kKeys + lane * p.box;
    if (lane < kKeys / p.box && pos < y.x.end && pos + p.box > y.x.lo) {
      const int at = pos / a.kv.page_size;
      x.off = pos - at * a.kv.page_size;
      x.entry = at < a.kv.max_pages ? a.kv.block_table[(long long)y.seq * a.kv.max_pages + at] : -1;
      if (x.entry < 0) x.entry = -1;
    }
    return x;
  };
  // slots: those of K, then those of V
  // (int8 cache: K is widened by the warps 4 n and 4 n + 1 from 8 on, V by 4 n + 2 and 4 n + 3 from
  // 14 on, so that the warps of a scheduler share their instructions)
  const bool loads_k = Q8 ? warp >= kSoftWarps && !(warp & 2) : warp == kKWarp, loads_v = Q8 ? warp > kQueryWarp && (warp & 2) : warp == kVWarp;
  if (loads_k || loads_v) {
    // ------------------------------------------------- the rings' loads
    const bool is_k = loads_k;
    const uint64_t policy = tc::policy_evict_last();
    const int nb = kKeys / p.box;                // boxes of a step's keys
    const int k_box0 = rank * (nb / 2);          // this CTA's half of them for K
    const int slots = is_k ? NKS : NVS, slot0 = is_k ? 0 : NKS, bytes = is_k ? S::kKSlot : S::kVSlot;
    const uint32_t base = is_k ? ring0 : v_ring0;
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    if constexpr (Q8) {
      const int cw = (warp - (is_k ? kSoftWarps : kQueryWarp + 3)) / 4 * 2 + (warp & 1), lg_box = 31 - __clz(p.box);
      // The steps' slots one after the other.
      auto run = [&](auto shape, auto two, auto key0, auto parts) {
        using W = decltype(shape);
        constexpr bool TWO = decltype(two)::value;
        constexpr int P = decltype(parts)::value, NB = P > 1 ? 2 : 1;   // slots (pairs of them) a step; how many are read ahead
        const int8_t* const codes = static_cast<const int8_t*>(TWO ? a.k : a.v) + W::piece(lane) * 16;
        const __half* const scales = static_cast<const __half*>(TWO ? a.k_scales : a.v_scales) + W::piece(lane) / 2;
        const int first_key = TWO ? rank * decltype(key0)::value : 0;
        auto dim_of = [&](int part, int h) { return TWO ? h * S::kKD : (part * 2 + rank) * (S::kN / 2); };
        const uint32_t p0 = W::place(cw, lane, 0), p1 = W::place(cw, lane, 1);
        W x[NB];
        StepRows st = {}, st2 = {};   // of this step and the next
        int part = 0, part2 = 0;
        auto plan_of = [&](int j, StepRows& to, int& part_to) {
          const bool f = wait_for<Q8>(tc::smem_u32(plan_bars + j % kPlans), (j / kPlans) & 1, p.wait_limit, abort_flag, p.dev_err);
          if (!__all_sync(0xffffffffu, f)) ok = false;
          const Plan& e = plans[j % kPlans];
          to = {ok ? e.row[lane & 7] : -1, e.k0, e.lo, e.end};
          part_to = ok ? e.part : 0;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(plan_bars + kPlans + j % kPlans));
        };
        int pairs = 0;
        // step -1 reads the first step's
#pragma unroll 1
        for (int j = -1; j < n_steps && ok; ++j) {
          if (j + 1 < n_steps) plan_of(j + 1, st2, part2);
#pragma unroll 1
          for (int h0 = 0; h0 < (j < 0 ? 1 : P); h0 += NB) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int h = h0 + i;
              if (j >= 0) {
                uint32_t at[2];
                int sl = slot;
                uint32_t rd = round;
                for (int k = 0; k < (TWO ? 2 : 1); ++k) {
                  at[k] = base + sl * bytes;
                  const bool f = ok && wait_for<Q8>(empty0 + 8 * (slot0 + sl), (rd & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err);
                  if (!__all_sync(0xffffffffu, f)) ok = false;
                  if (++sl == slots) sl = 0, ++rd;
                }
                if (!ok) continue;
#pragma unroll
                for (int u = 0; u < W::kGroups; ++u) x[i].template store<TWO>(at[0], at[TWO ? 1 : 0], p0, p1, cw, u, lane);
                tc::fence_proxy_async();
                __syncwarp();
                // (of two pieces, one barrier: the pair's number, mod the slots)
                if (lane == 0) tc::mbar_arrive_cluster(full0 + 8 * (slot0 + (TWO ? pairs : slot)), 0);
                if (++pairs == slots) pairs = 0;
                for (int k = 0; k < (TWO ? 2 : 1); ++k)
                  if (++slot == slots) slot = 0, ++round;
              }
              // (behind the stores: reads on their way would share what the stores wait by)
              const bool within = j >= 0 && h + NB < P;
              if (within || j + 1 < n_steps) {
                const StepRows from = within ? st : st2;
                const int dim = within ? dim_of(part, h + NB) : dim_of(part2, i);
#pragma unroll
                for (int u = 0; u < W::kGroups; ++u)
                  x[i].template load<!TWO>(codes + dim, scales + dim / 32, from, lg_box, first_key, cw, u, lane);
              }
            }
          }
          st = st2;
          part = part2;
        }
      };
      if (is_k) {
        run(Widen<kKeys / 2, S::kKD / 16, kWidenK, D>{}, std::true_type{}, std::integral_constant<int, kKeys / 2>{}, std::integral_constant<int, D / S::kKD>{});
      } else if (D == 64 && rank == 1) {   // columns beyond the head: zeros, once
        for (int j = 0; j < n_steps && ok; ++j) {
          const bool f = wait_for<Q8>(empty0 + 8 * (slot0 + slot), (round & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err);
          if (!__all_sync(0xffffffffu, f)) {
            ok = false;
            break;
          }
          if (round == 0) {
            for (int i = cw * 32 + lane; i < bytes / 16; i += kWidenV * 32)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + slot * bytes + i * 16), "r"(0) : "memory");
            tc::fence_proxy_async();
            __syncwarp();
          }
          if (lane == 0) tc::mbar_arrive_cluster(full0 + 8 * (slot0 + slot), 0);
          if (++slot == slots) slot = 0, ++round;
        }
      } else {
        run(Widen<kKeys, S::kN / 32, kWidenV, D>{}, std::false_type{}, std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
      }
    } else {
    Boxes next = {};
    if (n_steps > 0) next = fetch(w);
    for (int j = 0; j < n_steps && ok; ++j) {
      const Boxes cur = next;
      if (j + 1 < n_steps) {
        if (w.local + 1 < w.x.steps) ++w.local; else walk_next<PARTS>(w, p);
        next = fetch(w);
      }
      // the boxes' rows of the cache; total_rows, out of the cache, gives zeros
      const bool bad = cur.entry == -1 || cur.entry >= a.kv.n_pages;
      const int row = bad || cur.entry < 0 ? p.total_rows : (int)kv_row(a.kv, cur.entry, cur.head) + cur.off;
      const uint32_t mask = __ballot_sync(0xffffffffu, bad);
      if (is_k && lane == 0) {
        bad_sh[j % kBadRing] = mask;
        if (mask && a.err) *a.err = 1;
      }
      __syncwarp();
      const int n_slots = is_k ? S::kNK : 1;
      for (int h = 0; h < n_slots; ++h) {
        const uint32_t full = full0 + 8 * (slot0 + slot), dst = base + slot * bytes;
        const bool f = wait_for<Q8>(empty0 + 8 * (slot0 + slot), (round & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err);
        if (!__all_sync(0xffffffffu, f)) {
          ok = false;
          break;
        }
        if (lane == 0) tc::mbar_expect_tx(full, bytes);
        __syncwarp();
        if (is_k) {
          constexpr int slabs = S::kKD / 64;
          const int b = lane % (nb / 2), sl = lane / (nb / 2), r = __shfl_sync(0xffffffffu, row, k_box0 + b);
          if (sl < slabs) tc::tma_load_3d(dst + sl * (kKeys / 2 * 128) + b * p.box * 128, &p.tm_k, 0, r, h * slabs + sl, full, policy);
        } else {
          constexpr int slabs = S::kN / 128;   // this CTA's half of the columns (D = 64: the odd CTA's lie outside)
          const int b = lane % nb, sl = lane / nb, r = __shfl_sync(0xffffffffu, row, b);
          if (sl < slabs)
            tc::tma_load_3d(dst + sl * (kKeys * 128) + b * p.box * 128, &p.tm_v, 0, r, (cur.part * 2 + rank) * slabs + sl, full, policy);
        }
        if (++slot == slots) slot = 0, ++round;
      }
    }
    }
    // Before the CTA leaves, what was issued has landed and been used (that signal
    // may come from the other CTA): the slots of this round, and of the one before
    // those not yet filled again.
    for (int i = 0; i < slots; ++i) {
      const bool again = i < slot;
      if (!again && round == 0) continue;
      const uint32_t par = (again ? round : round - 1) & 1;
      const long long lim = *abort_flag ? kShortDrainCycles : kDrainCycles;
      if (!Q8) tc::mbar_drain(full0 + 8 * (slot0 + i), par, lim, p.dev_err);   // (widened: not by copies)
      tc::mbar_drain(empty0 + 8 * (slot0 + i), par, lim, p.dev_err);
    }
    __syncwarp();
  } else if (warp == kIssueWarp) {
    // -------------------------------------------------------- MMA issuer
    // The odd CTA's warp walks the same way and tells the even one what has landed.
    // (int8 cache: the warps that widen tell the even CTA themselves, and its issuing thread does
    // nothing else: every instruction between two MMAs waits its turn with five busy warps)
    constexpr uint32_t id_s = idesc(kKeys, BF16, false), id_o = idesc(S::kN, BF16, true);
    int ks = 0, vs = 0;                // slots
    uint32_t kround = 0, vround = 0;
    int item = 0;
    bool ok = n_steps > 0;
    if constexpr (Q8) {
      constexpr uint32_t kHighS = (uint32_t)(tc::desc_sw128(0) >> 32), kHighO = (uint32_t)(desc_mn_sw128(0, kKeys * 128) >> 32);
      if (rank == 1) {   // the queries' landing, item after item
#pragma unroll 1
        for (int j = 0; j < n_steps && ok; ++item) {
          ok = __all_sync(0xffffffffu, wait_for<Q8>(qfull, item & 1, p.wait_limit, abort_flag, p.dev_err));
          if (ok && lane == 0) tc::mbar_arrive_cluster(qfull, 0);
          j += w.x.steps - w.local;
          if (j < n_steps) walk_next<PARTS>(w, p);
        }
      } else if (tc::elect_one()) {
        int pairs = 0;
        uint32_t pround = 0;
        auto wait_one = [&](uint32_t bar, uint32_t par) {
          if (!wait_for<Q8>(bar, par, p.wait_limit, abort_flag, p.dev_err)) ok = false;
          return ok;
        };
        auto scores = [&](int j, bool first, bool last) {
          if (first && !wait_one(qfull, item & 1)) return;
          const uint32_t st = tmem + (j & 1) * 128;
          uint32_t qb = (uint32_t)tc::desc_sw128(q_addr);
#pragma unroll 1
          for (int h = 0; h < S::kNK / 2; ++h) {
            if (!wait_one(full0 + 8 * pairs, pround & 1)) return;
            tc::fence_after();
#pragma unroll 1
            for (int piece = 0; piece < 2; ++piece) {
              const uint32_t kb = (uint32_t)tc::desc_sw128(ring0 + ks * S::kKSlot);
#pragma unroll
              for (int k = 0; k < S::kKD / 16; ++k)
                mma_ss(st, qb + ((k >> 2) * (kRows * 128) + (k & 3) * 32) / 16, kb + ((k >> 2) * (kKeys / 2 * 128) + (k & 3) * 32) / 16,
                       kHighS, id_s, (h > 0 || piece > 0 || k > 0) ? 1u : 0u);
              tc::commit_pair(empty0 + 8 * ks);
              if (++ks == NKS) ks = 0;
            }
            qb += (S::kKD / 64) * (kRows * 128) / 16;
            if (++pairs == NKS) pairs = 0, ++pround;
          }
          tc::commit_pair(sfull0 + 8 * (j & 1));
          if (last) {
            tc::commit_pair(qempty);
            ++item;
          }
        };
        auto values = [&](int j, bool first) {
          if (!wait_one(pready0 + 8 * (j & 1), (j >> 1) & 1)) return;
          if (!wait_one(full0 + 8 * (NKS + vs), vround & 1)) return;
          tc::fence_after();
          const uint32_t vb = (uint32_t)desc_mn_sw128(v_ring0 + vs * S::kVSlot, kKeys * 128), pa = tmem + (j & 1) * 128;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k) {   // P of 32 keys lies over their scores: 16 columns, then the second piece's
            const uint32_t at = pa + 32 * (k >> 1) + 8 * (k & 1);
            mma_ts(o_tmem, at, vb + k * (2048 / 16), kHighO, id_o, (first && k == 0) ? 0u : 1u);
            if constexpr (SPLIT_P) mma_ts(o_tmem, at + 16, vb + k * (2048 / 16), kHighO, id_o, 1u);
          }
          tc::commit_pair(empty0 + 8 * (NKS + vs));   // also: O holds this step
          if (++vs == NVS) vs = 0, ++vround;
        };
        // one place each in the code: the next step's scores go before this one's values, those of
        // the next item behind them
        bool first = true, same = false;
#pragma unroll 1
        for (int j = -1; j < n_steps && ok; ++j) {
          const bool more = j + 1 < n_steps;
          bool next_has = false;
          if (more) {
            if (same) ++w.local; else if (j >= 0) walk_next<PARTS>(w, p);
            next_has = j + 2 < n_steps && w.local + 1 < w.x.steps;
          }
#pragma unroll 1
          for (int turn = 0; turn < 2 && ok; ++turn) {
            if ((turn == 0) == same) {
              if (more) scores(j + 1, !same, !next_has);
            } else if (j >= 0) {
              values(j, first);
            }
          }
          first = !same;
          same = next_has;
        }
      }
      __syncwarp();
    } else {
    auto wait_all = [&](uint32_t bar, uint32_t par) {
      const bool f = wait_for<Q8>(bar, par, p.wait_limit, abort_flag, p.dev_err);
      ok = __all_sync(0xffffffffu, f);
      if (ok && rank == 1 && lane == 0) tc::mbar_arrive_cluster(bar, 0);
      return ok;
    };
    auto scores = [&](int j, bool first, bool last) {
      if (first && !wait_all(qfull, item & 1)) return;
      for (int h = 0; h < S::kNK; ++h) {
        if (!wait_all(full0 + 8 * ks, kround & 1)) return;
        if (rank == 0) {
          tc::fence_after();
          if (tc::elect_one()) {
            const uint32_t kb = (uint32_t)tc::desc_sw128(ring0 + ks * S::kKSlot), qb = (uint32_t)tc::desc_sw128(q_addr + h * (S::kKD / 64) * (kRows * 128));
#pragma unroll
            for (int k = 0; k < S::kKD / 16; ++k)
              mma_ss(tmem + (j & 1) * 128, qb + ((k >> 2) * (kRows * 128) + (k & 3) * 32) / 16, kb + ((k >> 2) * (kKeys / 2 * 128) + (k & 3) * 32) / 16,
                     (uint32_t)(tc::desc_sw128(0) >> 32), id_s, (h > 0 || k > 0) ? 1u : 0u);
            tc::commit_pair(empty0 + 8 * ks);
          }
          __syncwarp();
        }
        if (++ks == NKS) ks = 0, ++kround;
      }
      if (rank == 0) {
        if (tc::elect_one()) {
          tc::commit_pair(sfull0 + 8 * (j & 1));
          if (last) tc::commit_pair(qempty);
        }
        __syncwarp();
      }
      if (last) ++item;
    };
    auto values = [&](int j, bool first) {
      if (rank == 0 && !wait_all(pready0 + 8 * (j & 1), (j >> 1) & 1)) return;
      if (!wait_all(full0 + 8 * (NKS + vs), vround & 1)) return;
      if (rank == 0) {
        tc::fence_after();
        if (tc::elect_one()) {
          const uint32_t vb = (uint32_t)desc_mn_sw128(v_ring0 + vs * S::kVSlot, kKeys * 128), pa = tmem + (j & 1) * 128;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(o_tmem, pa + 8 * k, vb + k * (2048 / 16), (uint32_t)(desc_mn_sw128(0, kKeys * 128) >> 32), id_o, (first && k == 0) ? 0u : 1u);
          tc::commit_pair(empty0 + 8 * (NKS + vs));   // also: O holds this step
        }
        __syncwarp();
      }
      if (++vs == NVS) vs = 0, ++vround;
    };
    // per step: whether it is the first of an item in this share, and whether the
    // next step belongs to the same item
    bool first = true, has = false;
    if (ok) {
      has = 1 < n_steps && w.local + 1 < w.x.steps;
      scores(0, true, !has);
    }
    for (int j = 0; j < n_steps && ok; ++j) {
      const bool same = has;
      bool next_has = false;
      if (j + 1 < n_steps) {
        if (same) ++w.local; else walk_next<PARTS>(w, p);
        next_has = j + 2 < n_steps && w.local + 1 < w.x.steps;
      }
      if (same) scores(j + 1, false, !next_has);
      if (ok) values(j, first);
      if (ok && !same && j + 1 < n_steps) scores(j + 1, true, !next_has);
      first = !same;
      has = next_has;
    }
    }
    // every tcgen05 operation has finished, in both CTAs, before TMEM is freed
    if (rank == 0 && tc::elect_one()) tc::commit_pair(drain);
    __syncwarp();
    tc::mbar_drain(drain, 0, *abort_flag ? kShortDrainCycles : kDrainCycles, p.dev_err);
    __syncwarp();
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------- query rows
    // (int8 cache: and the plans of the steps, two ahead of the queries, so that waiting for
    // the last item's scores holds up no plan)
    constexpr int kAhead = Q8 ? 2 : 0;
    int item = 0, item_step = 0;   // the next item and its first step
    Walk y = w;
    Boxes next = {};
    if (Q8 && n_steps > 0) next = fetch(y);
#pragma unroll 1
    for (int j = 0; j < n_steps + kAhead; ++j) {
      if (Q8 && j < n_steps) {
        const bool bad = next.entry == -1 || next.entry >= a.kv.n_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, bad);
        const int row = bad || next.entry < 0 ? -1 : (int)kv_row(a.kv, next.entry, next.head) + next.off;
        const int k0 = y.x.base + y.local * kKeys, lo = y.x.lo, end = y.x.end, part = next.part;
        if (j + 1 < n_steps) {   // the next step's table entries are on their way meanwhile
          if (y.local + 1 < y.x.steps) ++y.local; else walk_next<PARTS>(y, p);
          next = fetch(y);
        }
        const int at = j % kPlans;
        if (!__all_sync(0xffffffffu, wait_for<Q8>(tc::smem_u32(plan_bars + kPlans + at), ((j / kPlans) & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err)))
          break;
        if (lane < 8) plans[at].row[lane] = row;
        if (lane == 0) {
          plans[at].k0 = k0, plans[at].lo = lo, plans[at].end = end, plans[at].part = part;
          bad_sh[j % kBadRing] = mask;
          if (mask && a.err) *a.err = 1;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(plan_bars + at));
      }
      if (j - kAhead != item_step) continue;
      if (!__all_sync(0xffffffffu, wait_for<Q8>(qempty, (item & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err))) break;
      if (lane == 0) tc::mbar_expect_tx(qfull, (D / 64) * p.tokens * p.group * 128);
      __syncwarp();
      // tokens behind the sequence's are another's or, behind the last, zeros:
      // their rows are masked and not written
      if (lane < D / 64)
        tc::tma_load_4d(q_addr + lane * (kRows * 128), &p.tm_q, 0, w.head * p.group, w.s.cu + (2 * w.t + rank) * p.tokens, lane, qfull);
      ++item;
      item_step += w.x.steps - w.local;
      if (item_step < n_steps) walk_next<PARTS>(w, p);
    }
    // the loads land before the CTA leaves
    if (item > 0) tc::mbar_drain(qfull, (item - 1) & 1, *abort_flag ? kShortDrainCycles : kDrainCycles, p.dev_err);
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax
    const int row = threadIdx.x & (kRows - 1), half = warp >> 2;   // half of the step's keys, of O's columns
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // scores in units of log2 e; a scale of zero becomes one that still takes
    // the masked scores' infinity to infinity
    float sc = a.scale == 0.f ? 1e-30f : a.scale * 1.4426950408889634f;
    float m = -CUDART_INF_F, l = 0.f;
    // int8 cache: the reference lies `below` under the largest score, which is held unscaled (neg: with its sign
    // turned).  Differences of scores are then exact, and none passes the reference by more than `move`, however
    // large they are (of bf16 queries, up to 2^100): `most` is the magnitude where it moves, rounded down.  m, with
    // the rounding of an fp32 number of its size, is formed where a part or a log-sum is written.
    [[maybe_unused]] float neg = 0.f, most = -CUDART_INF_F;
    [[maybe_unused]] auto top_of = [&]() { return most == -CUDART_INF_F ? most : sc < 0.f ? neg : -neg; };
    bool first = true, opens = w.local == 0, dead = false;
    const int row_tok = row < p.tokens * p.group ? row / p.group : 1 << 28, row_head = row % p.group;
    int lo = 0, hi = -1, tok = 0;
    // the two warps of the same rows meet; a dead one too, so that none is left waiting
    auto meet = [&]() {
      tc::fence_before();
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
      tc::fence_after();
    };
    auto wait = [&](uint32_t bar, uint32_t par) {
      if (!dead) dead = !__all_sync(0xffffffffu, wait_for<Q8>(bar, par, p.wait_limit, abort_flag, p.dev_err));
      tc::fence_after();
    };
    // O holds step i: the MMAs that read its slot of V are complete
    auto wait_values = [&](int i) { wait(empty0 + 8 * (NKS + i % NVS), (i / NVS) & 1); };
    auto begin = [&]() {
      tok = (2 * w.t + rank) * p.tokens + row_tok;
      const int pos = tok < w.s.n ? w.s.pos0 + tok : -1;
      if constexpr (Q8) {
        if (p.row_scale) {
          sc = a.scale * 1.4426950408889634f * (tok < w.s.n ? p.row_scale[(long long)(w.s.cu + tok) * a.n_q + w.head * p.group + row_head] : 1.f);
          if (sc == 0.f) sc = 1e-30f;
        }
      }
      lo = kv_first(pos, a.window);
      hi = min(pos, w.x.end - 1);
      m = -CUDART_INF_F, l = 0.f;
      neg = 0.f, most = -CUDART_INF_F;
      first = true;
    };
    if (n_steps > 0) begin();
    constexpr int kHalfO = S::kDV / 2;
    const uint32_t o_half = o_tmem + lane_off + half * kHalfO;
#pragma unroll 1
    for (int j = 0; j < n_steps; ++j) {
      const int k0 = w.x.base + w.local * kKeys, kh = k0 + 64 * half;   // the step's keys, this thread's
      const bool same = j + 1 < n_steps && w.local + 1 < w.x.steps;
      const uint32_t s_tmem = tmem + lane_off + (j & 1) * 128;
      wait(sfull0 + 8 * (j & 1), (j >> 1) & 1);
      float s[Q8 ? 32 : 64];
      if constexpr (!Q8) tc::tmem_ld64(s_tmem + 64 * half, s);
      const uint32_t bad = bad_sh[j % kBadRing];
      // bit i: the row sees key kh + i
      [[maybe_unused]] uint32_t see0 = ~0u, see1 = ~0u;
      const float none = sc < 0.f ? CUDART_INF_F : -CUDART_INF_F;
      const bool masked = bad || kh < lo || kh + 63 > hi;
      if (masked) {
        auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
        unsigned long long see = below(hi + 1 - kh) & ~below(lo - kh);
        if (bad) {
          for (int i = 0; i < 64; i += 16)
            if ((bad >> ((64 * half + i) / p.box)) & 1) see &= ~(0xffffull << i);
        }
        see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
        if constexpr (!Q8) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = (see0 >> i) & 1 ? s[i] : none;
            s[32 + i] = (see1 >> i) & 1 ? s[32 + i] : none;
          }
        }
      }
      // int8 cache: 32 of the scores
      [[maybe_unused]] auto scores_of = [&](int h) {
        if constexpr (Q8) {
          tc::tmem_ld32(s_tmem + 64 * half + 32 * h, s);
          if (masked) {
            const uint32_t see = h ? see1 : see0;
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = (see >> i) & 1 ? s[i] : none;
          }
        }
      };
      // the maximum of scale * score: of the scores for a positive scale, of the
      // negated ones for a negative
      {
        float v[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
        constexpr int N = Q8 ? 32 : 64;
#pragma unroll 1
        for (int h = 0; h < 64 / N; ++h) {
          scores_of(h);
          if constexpr (Q8) {
            if (sc < 0.f) {
#pragma unroll
              for (int i = 0; i < N; ++i) s[i] = -s[i];
            }
#pragma unroll
            for (int i = 0; i < N; i += 2) v[(i >> 1) & 3] = max3(v[(i >> 1) & 3], s[i], s[i + 1]);
          } else if (sc >= 0.f) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i & 3] = fmaxf(v[i & 3], s[i]);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i & 3] = fmaxf(v[i & 3], -s[i]);
          }
        }
        float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        row_sh[half][j & 1][row] = Q8 || mx == -CUDART_INF_F ? mx : mx * fabsf(sc);
      }
      meet();
      const float mx = fmaxf(row_sh[0][j & 1][row], row_sh[1][j & 1][row]);   // (int8 cache: not scaled)
      if (__any_sync(0xffffffffu, mx > (Q8 ? most : m + Reference<P16>::move))) {
        float f;
        if constexpr (Q8) {
          const float top = top_of(), t2 = fmaxf(top, mx);
          f = 1.f;
          if (t2 > top) {
            f = ex2((top - t2) * fabsf(sc));
            neg = sc < 0.f ? t2 : -t2;
            most = __fadd_rd(t2, (Reference<P16>::move - Reference<P16>::below) / fabsf(sc));
          }
        } else {
          const float m2 = fmaxf(m, mx - Reference<P16>::below);
          f = m2 == -CUDART_INF_F ? 1.f : ex2(m - m2);
          m = m2;
        }
        l *= f;
        if (!first) {   // O holds the steps before: let the last one finish
          wait_values(j - 1);
#pragma unroll 1
          for (int c = 0; c < kHalfO; c += 32) {
            float t[32];
            uint32_t u[32];
            tc::tmem_ld32(o_half + c, t);
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(t[i] * f);
            tc::tmem_st32(o_half + c, u);
          }
        }
      }
      [[maybe_unused]] const float mb = m == -CUDART_INF_F ? 0.f : m;
      {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        [[maybe_unused]] f2_t pairs[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        constexpr int N = Q8 ? 16 : 32;
#pragma unroll 1
        for (int h = 0; h < 32 / N; ++h) {
          scores_of(h);
          uint32_t u[N];
          if constexpr (Q8) {
            const f2_t ref = f2_pack(neg, neg), by = f2_pack(sc, sc), add = f2_pack(Reference<P16>::below, Reference<P16>::below);
            constexpr int M = SPLIT_P ? 8 : N;   // pairs at once: two pieces of eight take the registers of one of 16
#pragma unroll
            for (int g = 0; g < N; g += M) {
              [[maybe_unused]] uint32_t v[8], rest[8];
#pragma unroll
              for (int i = g; i < g + M; ++i) {
                float x0, x1;
                f2_unpack(f2_fma(f2_add(f2_pack(s[2 * i], s[2 * i + 1]), ref), by, add), x0, x1);
                const float e0 = ex2(x0), e1 = ex2(x1);
                pairs[i & 1] = f2_add(pairs[i & 1], f2_pack(e0, e1));
                u[i] = Half16<P16>::pack(e0, e1);
                if constexpr (SPLIT_P) {
                  const float2 r = Half16<P16>::unpack(u[i]);
                  v[i - g] = u[i];
                  rest[i - g] = Half16<P16>::pack(e0 - r.x, e1 - r.y);
                }
              }
              if constexpr (SPLIT_P) {
                tc::tmem_st8(s_tmem + 64 * half + 32 * h + g, v);
                tc::tmem_st8(s_tmem + 64 * half + 32 * h + 16 + g, rest);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float e0 = ex2(fmaf(s[2 * i], sc, -mb)), e1 = ex2(fmaf(s[2 * i + 1], sc, -mb));
              sum[(2 * i) & 3] += e0;
              sum[(2 * i + 1) & 3] += e1;
              u[i] = Half16<P16>::pack(e0, e1);
            }
          }
          // P of the other half lies where this half's scores are: both have read
          // theirs (meet()).  (Int8 cache: over the 32 scores just read.)
          if constexpr (!Q8) tc::tmem_st32(s_tmem + 32 * half, u);
          else if constexpr (!SPLIT_P) tc::tmem_st16(s_tmem + 64 * half + 32 * h, u);
        }
        if constexpr (Q8) f2_unpack(pairs[0], sum[0], sum[1]), f2_unpack(pairs[1], sum[2], sum[3]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // values that no row of the tile sees may be anything, and 0 times
      // infinity is no zero: they are cleared in shared memory
      // (int8 cache: they are written as zeros)
      if (!Q8 && (k0 < w.x.lo || k0 + kKeys > w.x.end)) {
        // The parity tells two neighbouring phases apart.  With several slots the one
        // before has landed (its step is NVS back, and this step's scores were issued
        // after the values two steps back).  With one it is the step before, whose
        // values may still be on their way: they have been used first.
        if (NVS == 1 && j > 0) wait_values(j - 1);
        wait(full0 + 8 * (NKS + j % NVS), (j / NVS) & 1);
        const uint32_t vb = v_ring0 + j % NVS * S::kVSlot;
        // a thread clears one 16-byte piece of a row of every slab
        for (int i = threadIdx.x; i < kKeys * 8; i += kSoftWarps * 32) {
          const int c = k0 + (i >> 3);
          if (c < w.x.lo || c >= w.x.end) {
#pragma unroll
            for (int sl = 0; sl < S::kN / 128; ++sl)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + sl * (kKeys * 128) + i * 16), "r"(0) : "memory");
          }
        }
        tc::fence_proxy_async();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(pready0 + 8 * (j & 1), 0);
      first = false;
      if (same) {
        ++w.local;
        continue;
      }
      // ---- the item's part is complete.  The barrier's parity tells two
      // neighbouring phases apart, so the step before is waited for first (the
      // one before that is complete: this step's scores were issued after it).
      if (j > 0) wait_values(j - 1);
      wait_values(j);
      const bool closes = w.local + 1 == w.x.steps, whole = opens && closes;
      const bool in = tok < w.s.n && !dead;
      // the row's sum: of both halves
      row_sh[half][j & 1][row] = l;   // every maximum in it has been read: the step's products are complete
      meet();
      l = row_sh[0][j & 1][row] + row_sh[1][j & 1][row];
      if constexpr (Q8) m = top_of() * fabsf(sc) - Reference<P16>::below;
      const long long orow = (long long)(w.s.cu + tok) * a.n_q + w.head * p.group + row_head;
      const long long slot = (2ll * pair + (opens ? 1 : 0)) * 2 + rank;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* out = static_cast<T*>(a.out) + orow * D + w.part * S::kDV + half * kHalfO;
      float* po = p.split.part_o + (slot * S::kDV + half * kHalfO) * kRows + row * 4;
#pragma unroll 1
      for (int c = 0; c < kHalfO; c += 32) {
        float t[32];
        tc::tmem_ld32(o_half + c, t);
        if (!in) continue;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(out + c + i) =
                make_uint4(Half16<T>::pack(t[i] * inv, t[i + 1] * inv), Half16<T>::pack(t[i + 2] * inv, t[i + 3] * inv),
                           Half16<T>::pack(t[i + 4] * inv, t[i + 5] * inv), Half16<T>::pack(t[i + 6] * inv, t[i + 7] * inv));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(po + (c + i) * kRows) = make_float4(t[i], t[i + 1], t[i + 2], t[i + 3]);
        }
      }
      if (half == 0) {
        if (!whole) p.split.part_ml[slot * kRows + row] = make_float2(m, l);
        else if (in && w.part == 0 && a.lse) a.lse[orow] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
        if (opens && !closes && row == 0)
          p.split.recs[blockIdx.x] = {(int)((first_step + j - w.local + w.x.steps - 1) / share), w.s.cu + (2 * w.t + rank) * p.tokens,
                                      max(min(p.tokens, w.s.n - (2 * w.t + rank) * p.tokens), 0) * p.group, w.head * p.group, p.group, w.part};
      }
      tc::fence_before();
      if (j + 1 < n_steps) {
        walk_next<PARTS>(w, p);
        opens = true;
        begin();
      }
    }
  }

  // no CTA leaves while the other still loads into it or signals its barriers
  tc::fence_before();
  __syncwarp();
  tc::cluster_arrive_release();
  tc::cluster_wait();
  if (warp == kIssueWarp) {
    tc::fence_after();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

template <typename T, int D, bool Q8 = false>
static int launch(Params& p, const DeviceInfo& dev, cudaStream_t s) {
  using S = Shape<D, Q8>;
  static PerDevice attr;
  if (!attr.get(dev.ordinal)) {
    const cudaError_t e = cudaFuncSetAttribute(tile_kernel<T, D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "tile attention smem attribute");
    attr.set(dev.ordinal);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // as many pairs as the device holds at once (asked once per device)
  static int most[64] = {0};
  int n = dev.ordinal >= 0 && dev.ordinal < 64 ? most[dev.ordinal] : 0;
  if (n == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, tile_kernel<T, D, Q8>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "tile attention cluster occupancy");
    if (n < 1) return fail(Q4_ERR_CUDA, "tile attention: no cluster of two CTAs fits the device");
    if (dev.ordinal >= 0 && dev.ordinal < 64) most[dev.ordinal] = n;
  }
  if (n < p.pairs) p.pairs = n;
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_kernel<T, D, Q8>, p);
  if (e != cudaSuccess) return cuda_fail(e, "tile attention launch");
  return launch_attn_join(p.a, p.split, kRows, D, S::kDV, std::is_same<T, __nv_bfloat16>::value, 2 * p.pairs, 2, s);
}

}  // namespace tile
}  // namespace q4w
