// What the attention kernels share: the part of a sequence's work that its
// lengths determine, and the joining of parts that several CTAs had.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "q4w_internal.cuh"
#include "q4w_kv.cuh"

namespace q4w {

struct Seq {
  int n, pos0;           // new tokens taken, position of the first
  int base, end;         // keys [base, end) that any of them sees, base a multiple of `align`
  int cu;                // the first one's index
};

// align: a power of two that divides the page size.
__device__ __forceinline__ Seq seq_of(const AttnParams& a, int seq, int align) {
  Seq s;
  s.cu = a.kv.cu_tokens[seq];
  const int n = a.kv.cu_tokens[seq + 1] - s.cu, len = max(a.kv.kv_lens[seq], 0);
  s.n = s.cu >= 0 ? min(min(max(n, 0), a.max_q), max(a.T - s.cu, 0)) : 0;
  s.pos0 = len - n;
  s.base = kv_first(s.pos0, a.window) & ~(align - 1);
  s.end = s.n > 0 ? min(s.pos0 + s.n, a.kv.max_pages * a.kv.page_size) : 0;
  return s;
}
// More tokens than max_q, or a length that the block table does not hold.
__device__ __forceinline__ bool seq_bad(const AttnParams& a, int seq) {
  const int n = a.kv.cu_tokens[seq + 1] - a.kv.cu_tokens[seq];
  return n > a.max_q || (n > 0 && a.kv.kv_lens[seq] > a.kv.max_pages * a.kv.page_size);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where a row's running reference m lies (units of log2 e): it is set `below` under the
// maximum and moved when a score passes it by `move`, so that most steps rescale nothing.
// The probabilities 2^(s - m) enter the second product in 16 bits.  bf16 has the range of
// fp32.  fp16 has 30 octaves of normal numbers, and what is used of them above 1 is
// gained below: with m at the maximum a probability of 2^-20 kept four bits, and a
// hundred thousand keys of 2^-25 each were lost whole; now 2^-21 of the largest is a
// normal number and the absolute error 2^-32 of it.  2^15 fits, 65504 is the largest.
template <typename T>
struct Reference {
  static constexpr float below = std::is_same<T, __half>::value ? 7.f : 0.f, move = below + 8.f;
};

// The parts of work that is cut.  The steps of all items form one line that is
// cut into equal shares; the team of R CTAs c (R is 1, or 2 that work in step on
// a tile each) leaves the part of an item that began before it in slot 2 c, and
// the part of one that it begins and does not end in slot 2 c + 1, times R plus
// the CTA's rank, with a record per CTA of how far that item goes.
struct SplitRec {
  int last;              // team that ends the item; -1: this one begins none that it does not end
  int token, used;       // first token of the item's tile, its rows
  int head0, group;      // first query head, heads per token: row r is token r / group, head r % group
  int col;               // column part of D
};
struct AttnSplit {
  float* part_o;         // [2 grid][dv / 4][rows][4]: sums of the values
  float2* part_ml;       // [2 grid][rows]: reference (in units of log2 e) and sum
  SplitRec* recs;        // [grid]
};

inline size_t attn_up256(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t attn_split_bytes(int grid, int rows, int dv) {
  return attn_up256(grid * sizeof(SplitRec)) + attn_up256(2 * (size_t)grid * rows * sizeof(float2)) +
         attn_up256(2 * (size_t)grid * rows * dv * 4);
}
inline AttnSplit attn_split(void* ws, int grid, int rows, int dv) {
  AttnSplit s;
  char* w = static_cast<char*>(ws);
  s.recs = reinterpret_cast<SplitRec*>(w);
  w += attn_up256(grid * sizeof(SplitRec));
  s.part_ml = reinterpret_cast<float2*>(w);
  w += attn_up256(2 * (size_t)grid * rows * sizeof(float2));
  s.part_o = reinterpret_cast<float*>(w);
  return s;
}

// Joins what the recorded items left in their slots, in the order of the keys.
int launch_attn_join(const AttnParams& a, const AttnSplit& split, int rows, int D, int dv, bool bf16, int grid, int R,
                     cudaStream_t s);

}  // namespace q4w
