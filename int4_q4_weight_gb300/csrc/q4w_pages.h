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

}  // namespace q4w
