// What the paged-cache kernels share: the cache's layout and the lookups in
// its tables.  A cache is [n_pages][n_kv][page_size][head_dim] for K and for
// V, so the rows of one KV head inside a page are contiguous.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/q4w.h"
#include "q4w_pages.h"

namespace q4w {

constexpr int kMaxSeqs = 4096;

struct KvTables {
  const int32_t* block_table;   // [n_seqs][max_pages]
  const int32_t* cu_tokens;     // [n_seqs + 1]
  const int32_t* kv_lens;       // [n_seqs]
  int n_seqs, max_pages, n_pages, n_kv, page_size;
};

inline KvTables kv_tables(const q4_kv_cache& c) {
  return {c.block_table, c.cu_tokens, c.kv_lens, c.n_seqs, c.max_pages, c.n_pages, c.n_kv, c.page_size};
}

// Page of a position of sequence `seq`, or -1 (q4w_pages.h).
__device__ __forceinline__ int kv_page(const KvTables& t, int seq, int pos) {
  return kv_page(t.block_table + (long long)seq * t.max_pages, t.max_pages, t.n_pages, t.page_size, pos);
}
__device__ __forceinline__ long long kv_row(const KvTables& t, int page, int head) {
  return kv_row(page, t.n_kv, t.page_size, head);
}

// One attention call.
struct AttnParams {
  KvTables kv;
  const void *k, *v;        // the cache
  const void* q;            // [T][n_q][D], token stride in elements
  long long q_stride;
  void* out;                // [T][n_q][D]
  float* lse;               // [T][n_q] or NULL
  int32_t* err;
  int T, n_q, max_q, window;
  float scale;
};

struct DeviceInfo;
int launch_kv_append(const q4_kv_cache& c, int T, const void* k, long long k_stride, const void* v,
                     long long v_stride, int in_dtype, const void* q, long long q_stride, int n_q, void* q_out,
                     const uint64_t* steps, int rot, int interleaved, const int32_t* positions, int32_t* err,
                     const DeviceInfo& dev, cudaStream_t s);
// Workspace of an attention call whose sequences have up to max_rows query
// rows (tokens x query heads) per KV head.
size_t attn_ws_bytes(long long max_rows, int D, const DeviceInfo& dev);
// Tensor map of a cache of `rows` rows of D 16-bit elements, seen as D/64 slabs
// of 64 elements: boxes of box_rows rows of box_slabs slabs in the 128-byte
// swizzle, laid out slab after slab.
int encode_cache_rows(CUtensorMap* tm, const void* base, bool bf16, int D, uint64_t rows, uint32_t box_rows,
                      uint32_t box_slabs, const char* what);
// Query rows [T][n_q][D] of 16-bit elements with a token stride, as D/64 slabs:
// boxes of `tokens` tokens of `heads` heads of one slab, 128-byte swizzle.
int encode_query_rows(CUtensorMap* tm, const void* base, bool bf16, int D, int n_q, int T, long long stride,
                      uint32_t heads, uint32_t tokens);
// Few query rows per KV head (k_attn_decode.cu).
bool attn_decode_fits(long long max_rows, int D);
size_t attn_decode_ws_bytes(int max_rows, int D, const DeviceInfo& dev);
int launch_attn_decode(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s);
// Tiles of 128 query rows (k_attn_tile.cu).
size_t attn_tile_ws_bytes(int D, const DeviceInfo& dev);
int launch_attn_tile(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s);
int launch_kv_attention(const AttnParams& p, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s);

int launch_logits_sample(const void* z, long long stride, int dtype, int rows, int V, const float* u,
                         const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                         int32_t* token, float* logprob, const DeviceInfo& dev, cudaStream_t s);

// 16-bit float types of the cache: conversion from fp32 (nearest even) and to it.
template <typename T>
struct Half16;
template <>
struct Half16<__half> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
};
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};

}  // namespace q4w
