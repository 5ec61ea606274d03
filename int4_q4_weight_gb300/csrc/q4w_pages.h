// The paged cache's index arithmetic, plain C++ so that it also compiles for
// the host.  Every access of a kernel to a page goes through kv_page: what it
// returns is a page inside the cache or -1.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define Q4W_HD __host__ __device__ __forceinline__
#else
#define Q4W_HD inline
#endif

namespace q4w {

// Page that holds position `pos` of the sequence whose block-table row is
// `row`, or -1: a negative position, one behind the row, or an entry that is
// no page of the cache.
Q4W_HD int kv_page(const int32_t* row, int max_pages, int n_pages, int page_size, int pos) {
  if (pos < 0) return -1;
  const int at = pos / page_size;
  if (at >= max_pages) return -1;
  const int page = row[at];
  return page >= 0 && page < n_pages ? page : -1;
}

// First row (of n_pages * n_kv * page_size rows of head_dim elements) of KV
// head `head` in `page`.
Q4W_HD long long kv_row(int page, int n_kv, int page_size, int head) {
  return ((long long)page * n_kv + head) * page_size;
}

// First position that a token at `pos` sees with a window (0: all).  (The
// difference is only formed where it is positive: a large window and a negative
// position leave 32 bits.)
Q4W_HD int kv_first(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

// The keys that tile t (of `tokens` tokens) of a sequence sees: [base, end), base a
// multiple of `box` (a power of two), and its steps of kv_tile_keys keys; one step
// where it sees nothing.  The sequence: n new tokens, the first at pos0, keys below `end`.
constexpr int kv_tile_keys = 128;
struct KvSpan {
  int lo, base, end, steps;   // lo: the first key that its first token sees
};
Q4W_HD KvSpan kv_span(int pos0, int n, int end, int window, int tokens, int t, int box) {
  KvSpan x;
  const int j0 = t * tokens, j1 = (n - j0 < tokens ? n : j0 + tokens) - 1;
  x.lo = kv_first(pos0 + j0, window);
  x.base = x.lo & ~(box - 1);
  x.end = end < pos0 + j1 + 1 ? end : pos0 + j1 + 1;
  x.steps = x.end > x.base ? (x.end - x.base + kv_tile_keys - 1) / kv_tile_keys : 1;
  return x;
}
// Steps of the tiles first, first + stride, .. of a sequence: a tile has up to 2^24 and a
// sequence up to 2^24 tiles, so 64 bits.
Q4W_HD long long kv_tile_steps(int pos0, int n, int end, int window, int tokens, int box, int first, int stride) {
  long long sum = 0;
  for (long long t = first; t * tokens < n; t += stride) sum += kv_span(pos0, n, end, window, tokens, (int)t, box).steps;
  return sum;
}
// Steps of the share of `share` that begins at `first` of `total`; -1 where a share passes
// 32 bits: hours of work, which the kernels leave out and flag.
Q4W_HD int kv_share_steps(long long total, long long share, long long first) {
  if (share > 0x7fffffff) return -1;
  const long long n = total - first < share ? total - first : share;
  return n > 0 ? (int)n : 0;
}

}  // namespace q4w
