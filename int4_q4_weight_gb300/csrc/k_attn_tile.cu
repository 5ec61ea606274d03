// Attention of many query rows per KV head over a paged cache (prefill chunks,
// prompts): tiles of 128 query rows on the 5th-generation tensor cores.
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
#include <cuda.h>

#include "q4w_attn.cuh"
#include "q4w_device.cuh"
#include "q4w_tc_pair.cuh"

namespace q4w {
namespace tile {

constexpr int kRows = 128, kKeys = kv_tile_keys;
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps, kKWarp = kMmaWarp + 1, kVWarp = kKWarp + 1, kQWarp = kVWarp + 1;
constexpr int kThr = (kQWarp + 1) * 32;
constexpr long long kDrainCycles = 2000000000LL;
constexpr long long kShortDrainCycles = 4000000LL;   // aborting: copies in flight land well within this
constexpr int kBadRing = 16;

template <int D>
struct Shape {
  static constexpr int kDV = D < 256 ? D : 256;              // columns of O of an item
  static constexpr int kParts = D / kDV;                     // items per tile
  static constexpr int kN = D == 64 ? 128 : kDV;             // columns of the MMA (D = 64: the odd CTA's are zeros)
  static constexpr int kKD = D < 256 ? D : 256;              // dims of a K slot
  static constexpr int kNK = D / kKD;                        // K slots per step
  static constexpr int kKSlot = kKeys / 2 * kKD * 2;         // bytes: 8, 16, 32, 32 KB
  static constexpr int kVSlot = kKeys * kN;                  // all keys of a step, kN / 2 columns a CTA: 16, 16, 32, 32 KB
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKSlots = D <= 128 ? 6 : 2;           // rings of K and of V
  static constexpr int kVSlots = D <= 128 ? 6 : D == 256 ? 3 : 1;
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

// Instruction descriptor, kind::f16: fp32 accumulators, A and B of one 16-bit
// type, M = 256 (both CTAs' rows), N = n; bit 16: B is MN-major (its N index is the contiguous one).
__host__ __device__ constexpr uint32_t idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(2 * kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accum)
      : "memory");
}
// MN-major operand in the 128-byte swizzle: 64 elements of MN are one 128-byte
// row per K index, eight K rows (1024 bytes) a group (stride byte offset), the
// next 64 elements of MN `lbo` bytes further (leading byte offset).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
template <typename T, int D>
__global__ void __launch_bounds__(kThr, 1) tile_kernel(const __grid_constant__ Params p) {
  using S = Shape<D>;
  constexpr int NKS = S::kKSlots, NVS = S::kVSlots, NS = NKS + NVS, PARTS = S::kParts;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
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
      if (lane == 2 * NS + 4 || lane == 2 * NS + 5) count = rank == 0 ? 2 * kSoftWarps : 1;      // pready
      tc::mbar_init(tc::smem_u32(bars + lane), count);
    }
    tc::mbar_fence_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc_pair(tc::smem_u32(&tmem_sh), 512);
  if (lane == 0 && (warp == kKWarp || warp == kVWarp || warp == kQWarp)) {
    const CUtensorMap* m = warp == kKWarp ? &p.tm_k : warp == kVWarp ? &p.tm_v : &p.tm_q;
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

  // slots: those of K, then those of V
  if (warp == kKWarp || warp == kVWarp) {
    // ---------------------------------------------------------- TMA loads
    const bool is_k = warp == kKWarp;
    const uint64_t policy = tc::policy_evict_last();
    const int nb = kKeys / p.box;                // boxes of a step's keys
    const int k_box0 = rank * (nb / 2);          // this CTA's half of them for K
    const int slots = is_k ? NKS : NVS, slot0 = is_k ? 0 : NKS, bytes = is_k ? S::kKSlot : S::kVSlot;
    const uint32_t base = is_k ? ring0 : v_ring0;
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    // A step's boxes, lane b the box b: the block-table entry is fetched a step
    // before it is needed (the load takes longer than a slot's products).
    struct Boxes {
      int entry, off, head, part;   // entry -2: nothing to load
    };
    auto fetch = [&](const Walk& y) {
      Boxes x = {-2, 0, y.head, y.part};
      const int pos = y.x.base + y.local * kKeys + lane * p.box;
      if (lane < nb && pos < y.x.end && pos + p.box > y.x.lo) {
        const int at = pos / a.kv.page_size;
        x.off = pos - at * a.kv.page_size;
        x.entry = at < a.kv.max_pages ? a.kv.block_table[(long long)y.seq * a.kv.max_pages + at] : -1;
        if (x.entry < 0) x.entry = -1;
      }
      return x;
    };
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
        const bool f = tc::mbar_wait(empty0 + 8 * (slot0 + slot), (round & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err);
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
    // Before the CTA leaves, what was issued has landed and been used (that signal
    // may come from the other CTA): the slots of this round, and of the one before
    // those not yet filled again.
    for (int i = 0; i < slots; ++i) {
      const bool again = i < slot;
      if (!again && round == 0) continue;
      const uint32_t par = (again ? round : round - 1) & 1;
      const long long lim = *abort_flag ? kShortDrainCycles : kDrainCycles;
      tc::mbar_drain(full0 + 8 * (slot0 + i), par, lim, p.dev_err);
      tc::mbar_drain(empty0 + 8 * (slot0 + i), par, lim, p.dev_err);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------- MMA issuer
    // The odd CTA's warp walks the same way and tells the even one what has landed.
    constexpr uint32_t id_s = idesc(kKeys, BF16, false), id_o = idesc(S::kN, BF16, true);
    int ks = 0, vs = 0;                // slots
    uint32_t kround = 0, vround = 0;
    int item = 0;
    bool ok = n_steps > 0;
    auto wait_all = [&](uint32_t bar, uint32_t par) {
      const bool f = tc::mbar_wait(bar, par, p.wait_limit, abort_flag, p.dev_err);
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
            const uint32_t kb = ring0 + ks * S::kKSlot, qb = q_addr + h * (S::kKD / 64) * (kRows * 128);
#pragma unroll
            for (int k = 0; k < S::kKD / 16; ++k)
              mma_ss(tmem + (j & 1) * 128, tc::desc_sw128(qb + (k >> 2) * (kRows * 128) + (k & 3) * 32),
                     tc::desc_sw128(kb + (k >> 2) * (kKeys / 2 * 128) + (k & 3) * 32), id_s, (h > 0 || k > 0) ? 1u : 0u);
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
          const uint32_t vb = v_ring0 + vs * S::kVSlot, pa = tmem + (j & 1) * 128;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(o_tmem, pa + 8 * k, desc_mn_sw128(vb + k * 2048, kKeys * 128), id_o, (first && k == 0) ? 0u : 1u);
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
    // every tcgen05 operation has finished, in both CTAs, before TMEM is freed
    if (rank == 0 && tc::elect_one()) tc::commit_pair(drain);
    __syncwarp();
    tc::mbar_drain(drain, 0, *abort_flag ? kShortDrainCycles : kDrainCycles, p.dev_err);
    __syncwarp();
  } else if (warp >= kQWarp) {
    // ------------------------------------------------------- query rows
    int item = 0;
    for (int j = 0; j < n_steps; ++item) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(qempty, (item & 1) ^ 1, p.wait_limit, abort_flag, p.dev_err))) break;
      if (lane == 0) tc::mbar_expect_tx(qfull, (D / 64) * p.tokens * p.group * 128);
      __syncwarp();
      // tokens behind the sequence's are another's or, behind the last, zeros:
      // their rows are masked and not written
      if (lane < D / 64)
        tc::tma_load_4d(q_addr + lane * (kRows * 128), &p.tm_q, 0, w.head * p.group, w.s.cu + (2 * w.t + rank) * p.tokens, lane, qfull);
      j += w.x.steps - w.local;
      if (j < n_steps) walk_next<PARTS>(w, p);
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
    const float sc = a.scale == 0.f ? 1e-30f : a.scale * 1.4426950408889634f;
    float m = -CUDART_INF_F, l = 0.f;
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
      if (!dead) dead = !__all_sync(0xffffffffu, tc::mbar_wait(bar, par, p.wait_limit, abort_flag, p.dev_err));
      tc::fence_after();
    };
    // O holds step i: the MMAs that read its slot of V are complete
    auto wait_values = [&](int i) { wait(empty0 + 8 * (NKS + i % NVS), (i / NVS) & 1); };
    auto begin = [&]() {
      tok = (2 * w.t + rank) * p.tokens + row_tok;
      const int pos = tok < w.s.n ? w.s.pos0 + tok : -1;
      lo = kv_first(pos, a.window);
      hi = min(pos, w.x.end - 1);
      m = -CUDART_INF_F, l = 0.f;
      first = true;
    };
    if (n_steps > 0) begin();
    constexpr int kHalfO = S::kDV / 2;
    const uint32_t o_half = o_tmem + lane_off + half * kHalfO;
    for (int j = 0; j < n_steps; ++j) {
      const int k0 = w.x.base + w.local * kKeys, kh = k0 + 64 * half;   // the step's keys, this thread's
      const bool same = j + 1 < n_steps && w.local + 1 < w.x.steps;
      const uint32_t s_tmem = tmem + lane_off + (j & 1) * 128;
      wait(sfull0 + 8 * (j & 1), (j >> 1) & 1);
      float s[64];
      tc::tmem_ld64(s_tmem + 64 * half, s);
      const uint32_t bad = bad_sh[j % kBadRing];
      if (bad || kh < lo || kh + 63 > hi) {
        // bit i: the row sees key kh + i
        auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
        unsigned long long see = below(hi + 1 - kh) & ~below(lo - kh);
        if (bad) {
          for (int i = 0; i < 64; i += 16)
            if ((bad >> ((64 * half + i) / p.box)) & 1) see &= ~(0xffffull << i);
        }
        const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
        const float none = sc < 0.f ? CUDART_INF_F : -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = (see0 >> i) & 1 ? s[i] : none;
          s[32 + i] = (see1 >> i) & 1 ? s[32 + i] : none;
        }
      }
      // the maximum of scale * score: of the scores for a positive scale, of the
      // negated ones for a negative
      {
        float v[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
        if (sc >= 0.f) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i & 3] = fmaxf(v[i & 3], s[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i & 3] = fmaxf(v[i & 3], -s[i]);
        }
        float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        row_sh[half][j & 1][row] = mx == -CUDART_INF_F ? mx : mx * fabsf(sc);
      }
      meet();
      const float mx = fmaxf(row_sh[0][j & 1][row], row_sh[1][j & 1][row]);
      if (__any_sync(0xffffffffu, mx > m + Reference<T>::move)) {
        const float m2 = fmaxf(m, mx - Reference<T>::below), f = m2 == -CUDART_INF_F ? 1.f : ex2(m - m2);
        m = m2;
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
      const float mb = m == -CUDART_INF_F ? 0.f : m;
      {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float e0 = ex2(fmaf(s[2 * i], sc, -mb)), e1 = ex2(fmaf(s[2 * i + 1], sc, -mb));
          sum[(2 * i) & 3] += e0;
          sum[(2 * i + 1) & 3] += e1;
          u[i] = Half16<T>::pack(e0, e1);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // P of the other half lies where this half's scores are: both have read
        // theirs (meet())
        tc::tmem_st32(s_tmem + 32 * half, u);
      }
      // values that no row of the tile sees may be anything, and 0 times
      // infinity is no zero: they are cleared in shared memory
      if (k0 < w.x.lo || k0 + kKeys > w.x.end) {
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
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

template <typename T, int D>
static int launch(Params& p, const DeviceInfo& dev, cudaStream_t s) {
  using S = Shape<D>;
  static PerDevice attr;
  if (!attr.get(dev.ordinal)) {
    const cudaError_t e = cudaFuncSetAttribute(tile_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "tile attention smem attribute");
    attr.set(dev.ordinal);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(kThr);
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
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, tile_kernel<T, D>, &cfg);
    if (e != cudaSuccess) return cuda_fail(e, "tile attention cluster occupancy");
    if (n < 1) return fail(Q4_ERR_CUDA, "tile attention: no cluster of two CTAs fits the device");
    if (dev.ordinal >= 0 && dev.ordinal < 64) most[dev.ordinal] = n;
  }
  if (n < p.pairs) p.pairs = n;
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_kernel<T, D>, p);
  if (e != cudaSuccess) return cuda_fail(e, "tile attention launch");
  return launch_attn_join(p.a, p.split, kRows, D, S::kDV, std::is_same<T, __nv_bfloat16>::value, 2 * p.pairs, 2, s);
}

template <typename T>
static int launch_t(Params& p, int D, const DeviceInfo& dev, cudaStream_t s) {
  switch (D) {
    case 64: return launch<T, 64>(p, dev, s);
    case 128: return launch<T, 128>(p, dev, s);
    case 256: return launch<T, 256>(p, dev, s);
    default: return launch<T, 512>(p, dev, s);
  }
}

}  // namespace tile

size_t attn_tile_ws_bytes(int D, const DeviceInfo& dev) { return attn_split_bytes(dev.sms, tile::kRows, D < 256 ? D : 256); }

int launch_attn_tile(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  tile::Params p = {};
  const bool bf16 = c.dtype == Q4_BF16;
  const uint64_t rows = (uint64_t)c.n_pages * c.n_kv * c.page_size;
  p.box = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : 16;
  int st = encode_cache_rows(&p.tm_k, c.k, bf16, c.head_dim, rows, p.box, 1, "the K cache");
  if (st == Q4_OK) st = encode_cache_rows(&p.tm_v, c.v, bf16, c.head_dim, rows, p.box, 1, "the V cache");
  p.group = a.n_q / c.n_kv;
  p.tokens = tile::kRows / p.group;
  if (st == Q4_OK) st = encode_query_rows(&p.tm_q, a.q, bf16, c.head_dim, a.n_q, a.T, a.q_stride, p.group, p.tokens);
  if (st != Q4_OK) return st;
  p.a = a;
  p.pairs = dev.sms / 2;
  p.total_rows = (int)rows;
  p.wait_limit = wait_limit();
  p.dev_err = device_error_word();
  p.split = attn_split(ws, dev.sms, tile::kRows, c.head_dim < 256 ? c.head_dim : 256);
  return bf16 ? tile::launch_t<__nv_bfloat16>(p, c.head_dim, dev, s) : tile::launch_t<__half>(p, c.head_dim, dev, s);
}

}  // namespace q4w
