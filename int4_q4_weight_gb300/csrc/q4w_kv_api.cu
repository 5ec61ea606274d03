// C ABI of the paged cache, the attention over it and the sampling: argument
// checks, status codes, dispatch to launchers.
#include "q4w_internal.cuh"
#include "q4w_kv.cuh"

using namespace q4w;

#define CHECK_NULL(p)                                              \
  do {                                                             \
    if ((p) == nullptr) return fail(Q4_ERR_NULL, "%s is NULL", #p); \
  } while (0)
#define CHECK_ALIGN(p)                                                                   \
  do {                                                                                   \
    if ((p) != nullptr && !aligned16(p))                                                 \
      return fail(Q4_ERR_ALIGN, "%s (%p) is not 16-byte aligned", #p, (const void*)(p)); \
  } while (0)
#define CHECK(cond, ...)                                 \
  do {                                                   \
    if (!(cond)) return fail(Q4_ERR_SHAPE, __VA_ARGS__); \
  } while (0)
#define DEVICE_OR_RETURN(dev)       \
  DeviceInfo dev;                   \
  do {                              \
    int st_ = current_device(&dev); \
    if (st_ != Q4_OK) return st_;   \
  } while (0)

extern "C" {

// What kv_append and kv_attention ask of a cache alike.
static int check_cache(const q4_kv_cache* cache) {
  CHECK_NULL(cache);
  CHECK_NULL(cache->k);
  CHECK_NULL(cache->v);
  CHECK_NULL(cache->block_table);
  CHECK_NULL(cache->cu_tokens);
  CHECK_NULL(cache->kv_lens);
  CHECK_ALIGN(cache->k);
  CHECK_ALIGN(cache->v);
  CHECK_ALIGN(cache->block_table);
  CHECK_ALIGN(cache->cu_tokens);
  CHECK_ALIGN(cache->kv_lens);
  CHECK(cache->dtype == Q4_F16 || cache->dtype == Q4_BF16, "cache dtype=%d must be Q4_F16 or Q4_BF16", cache->dtype);
  const int d = cache->head_dim;
  CHECK(d == 64 || d == 128 || d == 256 || d == 512, "head_dim=%d must be 64, 128, 256 or 512", d);
  CHECK(cache->page_size >= 16 && cache->page_size <= 1024 && cache->page_size % 16 == 0,
        "page_size=%d must be a multiple of 16 in [16, 1024]", cache->page_size);
  CHECK(cache->n_pages >= 1, "n_pages=%d must be >= 1", cache->n_pages);
  CHECK(cache->n_kv >= 1 && cache->n_kv <= 1024, "n_kv=%d must be in [1, 1024]", cache->n_kv);
  CHECK(cache->n_seqs >= 1 && cache->n_seqs <= kMaxSeqs, "n_seqs=%d must be in [1, %d]", cache->n_seqs, kMaxSeqs);
  CHECK(cache->max_pages >= 1, "max_pages=%d must be >= 1", cache->max_pages);
  // rows of the cache and positions of a sequence are indexed in 32 bits
  CHECK((long long)cache->n_pages * cache->n_kv * cache->page_size < (1ll << 31),
        "n_pages * n_kv * page_size must be below 2^31");
  CHECK((long long)cache->max_pages * cache->page_size <= (1ll << 31) - 8192,
        "max_pages * page_size must be at most 2^31 - 8192");
  return Q4_OK;
}

static int check_stride(long long stride, long long least, int esize, const char* name) {
  CHECK(stride >= least && stride < (1ll << 40), "%s=%lld must be at least %lld", name, stride, least);
  if (stride * esize % 16) return fail(Q4_ERR_ALIGN, "%s=%lld elements is not a multiple of 16 bytes", name, stride);
  return Q4_OK;
}

// Everything that the appending calls check alike, then the launch.
static int append_checked(const KvAppend& a, q4_stream_t stream) {
  const q4_kv_cache* cache = &a.cache;
  int st = Q4_OK;
  const void *k = a.k, *v = a.v, *q = a.q, *q_out = a.q_out, *steps = a.steps, *positions = a.positions, *err = a.err;
  const void *q_norm = a.q_norm, *k_norm = a.k_norm, *v_norm = a.v_norm;
  const int T = a.T, n_q = a.n_q, rot_dim = a.rot, in_dtype = a.in_dtype, interleaved = a.interleaved;
  CHECK_NULL(k);
  CHECK_NULL(v);
  CHECK_ALIGN(k);
  CHECK_ALIGN(v);
  CHECK_ALIGN(q);
  CHECK_ALIGN(q_out);
  CHECK_ALIGN(steps);
  CHECK_ALIGN(positions);
  CHECK_ALIGN(q_norm);
  CHECK_ALIGN(k_norm);
  CHECK_ALIGN(v_norm);
  CHECK_ALIGN(err);
  CHECK(T >= 1, "T=%d must be >= 1", T);
  CHECK(in_dtype == Q4_F32 || in_dtype == Q4_F16 || in_dtype == Q4_BF16, "in_dtype=%d unknown", in_dtype);
  CHECK((q == nullptr) == (q_out == nullptr), "q and q_out must be given together");
  CHECK(q == nullptr || (n_q >= 1 && n_q <= 131072), "n_q=%d must be in [1, 131072]", n_q);
  CHECK(rot_dim >= 0 && rot_dim <= cache->head_dim && rot_dim % 16 == 0,
        "rot_dim=%d must be a multiple of 16 in [0, %d]", rot_dim, cache->head_dim);
  if (rot_dim > 0) CHECK_NULL(steps);
  CHECK(interleaved == 0 || interleaved == 1, "interleaved=%d must be 0 or 1", interleaved);
  CHECK(q_norm == nullptr || q != nullptr, "q_norm without q");
  CHECK(a.eps >= 0.f && a.eps <= 3.4e38f, "eps=%g must be finite and not negative", (double)a.eps);
  const int esize = in_dtype == Q4_F32 ? 4 : 2;
  const long long kv_row = (long long)cache->n_kv * cache->head_dim;
  if ((st = check_stride(a.k_stride, kv_row, esize, "k_stride")) != Q4_OK) return st;
  if ((st = check_stride(a.v_stride, kv_row, esize, "v_stride")) != Q4_OK) return st;
  if (q && (st = check_stride(a.q_stride, (long long)n_q * cache->head_dim, esize, "q_stride")) != Q4_OK) return st;
  DEVICE_OR_RETURN(dev);
  KvAppend c = a;
  if (!q) c.n_q = 0;
  return launch_kv_append(c, dev, reinterpret_cast<cudaStream_t>(stream));
}

int kv_append(const q4_kv_cache* cache, int T, const void* k, long long k_stride, const void* v, long long v_stride,
              int in_dtype, const void* q, long long q_stride, int n_q, void* q_out, const uint64_t* steps,
              int rot_dim, int interleaved, const int32_t* positions, int32_t* err, q4_stream_t stream) {
  clear_error();
  int st = check_cache(cache);
  if (st != Q4_OK) return st;
  return append_checked({*cache, nullptr, nullptr, T, k, k_stride, v, v_stride, in_dtype, q, q_stride, n_q, q_out, steps,
                         rot_dim, interleaved, positions, nullptr, nullptr, nullptr, 0.f, err},
                        stream);
}

int kv_append_norm(const q4_kv_cache* cache, int T, const void* k, long long k_stride, const void* v, long long v_stride,
                   int in_dtype, const void* q, long long q_stride, int n_q, void* q_out, const float* q_norm,
                   const float* k_norm, const float* v_norm, float eps, const uint64_t* steps, int rot_dim,
                   int interleaved, const int32_t* positions, int32_t* err, q4_stream_t stream) {
  clear_error();
  int st = check_cache(cache);
  if (st != Q4_OK) return st;
  return append_checked({*cache, nullptr, nullptr, T, k, k_stride, v, v_stride, in_dtype, q, q_stride, n_q, q_out, steps,
                         rot_dim, interleaved, positions, q_norm, k_norm, v_norm, eps, err},
                        stream);
}

static int check_cache_q8(const q4_kv_cache_q8* cache) {
  CHECK_NULL(cache);
  int st = check_cache(&cache->c);
  if (st != Q4_OK) return st;
  CHECK_NULL(cache->k_scales);
  CHECK_NULL(cache->v_scales);
  CHECK_ALIGN(cache->k_scales);
  CHECK_ALIGN(cache->v_scales);
  return Q4_OK;
}

int kv_append_q8(const q4_kv_cache_q8* cache, int T, const void* k, long long k_stride, const void* v,
                 long long v_stride, int in_dtype, const void* q, long long q_stride, int n_q, void* q_out,
                 const float* q_norm, const float* k_norm, const float* v_norm, float eps, const uint64_t* steps,
                 int rot_dim, int interleaved, const int32_t* positions, int32_t* err, q4_stream_t stream) {
  clear_error();
  int st = check_cache_q8(cache);
  if (st != Q4_OK) return st;
  return append_checked({cache->c, cache->k_scales, cache->v_scales, T, k, k_stride, v, v_stride, in_dtype, q, q_stride,
                         n_q, q_out, steps, rot_dim, interleaved, positions, q_norm, k_norm, v_norm, eps, err},
                        stream);
}

int kv_read_q8(const q4_kv_cache_q8* cache, int T, void* k_out, void* v_out, int32_t* err, q4_stream_t stream) {
  clear_error();
  int st = check_cache_q8(cache);
  if (st != Q4_OK) return st;
  CHECK_NULL(k_out);
  CHECK_NULL(v_out);
  CHECK_ALIGN(k_out);
  CHECK_ALIGN(v_out);
  CHECK_ALIGN(err);
  CHECK(T >= 1, "T=%d must be >= 1", T);
  CHECK((long long)T * cache->c.n_kv < (1ll << 31), "T * n_kv must be below 2^31");
  DEVICE_OR_RETURN(dev);
  return launch_kv_read_q8(*cache, T, k_out, v_out, err, reinterpret_cast<cudaStream_t>(stream));
}

size_t kv_attention_ws_bytes(int max_q, int n_q, int n_kv, int head_dim) {
  DeviceInfo dev;
  if (max_q < 1 || n_kv < 1 || n_q < n_kv || head_dim < 1 || current_device(&dev) != Q4_OK) return 0;
  return attn_ws_bytes((long long)max_q * (n_q / n_kv), head_dim, dev);
}

// What kv_attention and kv_attention_q8 check alike behind their caches; need: the workspace.
static int check_attention(const q4_kv_cache* cache, const AttnParams& p) {
  const void *q = p.q, *out = p.out, *lse_opt = p.lse, *err = p.err;
  const int T = p.T, max_q = p.max_q, n_q = p.n_q, window = p.window;
  CHECK_NULL(q);
  CHECK_NULL(out);
  CHECK_ALIGN(q);
  CHECK_ALIGN(out);
  CHECK_ALIGN(lse_opt);
  CHECK_ALIGN(err);
  CHECK(T >= 1, "T=%d must be >= 1", T);
  CHECK(max_q >= 1 && max_q <= T, "max_q=%d must be in [1, T=%d]", max_q, T);
  CHECK(n_q >= 1 && n_q % cache->n_kv == 0 && n_q / cache->n_kv <= 128,
        "n_q=%d must be a multiple of n_kv=%d, at most 128 times it", n_q, cache->n_kv);
  CHECK((long long)T * n_q < (1ll << 31), "T * n_q must be below 2^31");
  CHECK(window >= 0, "window=%d must be >= 0", window);
  CHECK(p.scale >= -3.4e38f && p.scale <= 3.4e38f, "scale=%g must be finite", (double)p.scale);
  return check_stride(p.q_stride, (long long)n_q * cache->head_dim, 2, "q_stride");
}

static int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need > 0 && (ws == nullptr || ws_bytes < need))
    return fail(Q4_ERR_WORKSPACE, "ws must hold %zu bytes (got %zu)", need, ws ? ws_bytes : (size_t)0);
  return Q4_OK;
}

int kv_attention(const q4_kv_cache* cache, int T, int max_q, const void* q, long long q_stride, int n_q, float scale,
                 int window, void* out, float* lse_opt, int32_t* err, void* ws, size_t ws_bytes, q4_stream_t stream) {
  clear_error();
  int st = check_cache(cache);
  if (st != Q4_OK) return st;
  const AttnParams p = {kv_tables(*cache), cache->k, cache->v, q, q_stride, out, lse_opt, err, T, n_q, max_q, window,
                        scale, nullptr, nullptr};
  if ((st = check_attention(cache, p)) != Q4_OK) return st;
  CHECK_ALIGN(ws);
  DEVICE_OR_RETURN(dev);
  if ((st = check_ws(ws, ws_bytes, attn_ws_bytes((long long)max_q * (n_q / cache->n_kv), cache->head_dim, dev))) != Q4_OK) return st;
  return launch_kv_attention(p, *cache, ws, dev, reinterpret_cast<cudaStream_t>(stream));
}

size_t kv_attention_q8_ws_bytes(int T, int max_q, int n_q, int n_kv, int head_dim) {
  DeviceInfo dev;
  if (T < 0 || max_q < 1 || n_kv < 1 || n_q < n_kv || head_dim < 1 || current_device(&dev) != Q4_OK) return 0;
  return attn_q8_ws_bytes(T, n_q, (long long)max_q * (n_q / n_kv), head_dim, dev);
}

int kv_attention_q8(const q4_kv_cache_q8* cache, int T, int max_q, const void* q, long long q_stride, int n_q,
                    float scale, int window, void* out, float* lse_opt, int32_t* err, void* ws, size_t ws_bytes,
                    q4_stream_t stream) {
  clear_error();
  int st = check_cache_q8(cache);
  if (st != Q4_OK) return st;
  const q4_kv_cache& c = cache->c;
  const AttnParams p = {kv_tables(c), c.k, c.v, q, q_stride, out, lse_opt, err, T, n_q, max_q, window,
                        scale, cache->k_scales, cache->v_scales};
  if ((st = check_attention(&c, p)) != Q4_OK) return st;
  CHECK_ALIGN(ws);
  DEVICE_OR_RETURN(dev);
  const int rows_of = c.dtype == Q4_BF16 ? T : 0;   // fp16 queries are read as they are
  if ((st = check_ws(ws, ws_bytes, attn_q8_ws_bytes(rows_of, n_q, (long long)max_q * (n_q / c.n_kv), c.head_dim, dev))) != Q4_OK) return st;
  return launch_kv_attention_q8(p, c, ws, dev, reinterpret_cast<cudaStream_t>(stream));
}

int logits_sample(const void* logits, long long stride, int dtype, int b, int V, const float* u,
                  const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                  int32_t* token, float* logprob_opt, q4_stream_t stream) {
  clear_error();
  CHECK_NULL(logits);
  CHECK_NULL(u);
  CHECK_NULL(token);
  CHECK_ALIGN(logits);
  CHECK_ALIGN(u);
  CHECK_ALIGN(temperature);
  CHECK_ALIGN(top_k);
  CHECK_ALIGN(top_p);
  CHECK_ALIGN(min_p);
  CHECK_ALIGN(token);
  CHECK_ALIGN(logprob_opt);
  CHECK(dtype == Q4_F32 || dtype == Q4_F16 || dtype == Q4_BF16, "dtype=%d unknown", dtype);
  CHECK(b >= 1 && b <= 65535, "b=%d must be in [1, 65535]", b);
  CHECK(V >= 1 && V <= 1048576, "V=%d must be in [1, 1048576]", V);
  CHECK(stride >= V && stride < (1ll << 40), "stride=%lld must be at least V=%d", stride, V);
  DEVICE_OR_RETURN(dev);
  return launch_logits_sample(logits, stride, dtype, b, V, u, temperature, top_k, top_p, min_p, token, logprob_opt,
                              dev, reinterpret_cast<cudaStream_t>(stream));
}

static bool draft_sizes_ok(int b, int k, int V) { return b >= 1 && b <= 65535 && k >= 0 && k <= 64 && V >= 1 && V <= 1048576; }

size_t draft_verify_ws_bytes(int b, int k, int V) { return draft_sizes_ok(b, k, V) ? draft_verify_bytes(b, k, V) : 0; }

int draft_verify(const void* logits, long long user_stride, long long row_stride, int dtype, int b, int k, int V,
                 const int32_t* drafts, const float* u, const void* draft_logits, long long draft_user_stride,
                 long long draft_row_stride, const float* temperature, int32_t* tokens, int32_t* accepted,
                 float* logprobs_opt, void* ws, size_t ws_bytes, q4_stream_t stream) {
  clear_error();
  CHECK_NULL(logits);
  CHECK_NULL(u);
  CHECK_NULL(tokens);
  CHECK_NULL(accepted);
  CHECK(dtype == Q4_F32 || dtype == Q4_F16 || dtype == Q4_BF16, "dtype=%d unknown", dtype);
  CHECK(b >= 1 && b <= 65535, "b=%d must be in [1, 65535]", b);
  CHECK(k >= 0 && k <= 64, "k=%d must be in [0, 64]", k);
  CHECK(V >= 1 && V <= 1048576, "V=%d must be in [1, 1048576]", V);
  if (k > 0) CHECK_NULL(drafts);
  // a row of logits may begin anywhere
  const uintptr_t esize = dtype == Q4_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % esize) return fail(Q4_ERR_ALIGN, "logits (%p) is not aligned to its type", logits);
  if (reinterpret_cast<uintptr_t>(draft_logits) % esize)
    return fail(Q4_ERR_ALIGN, "draft_logits (%p) is not aligned to its type", draft_logits);
  CHECK_ALIGN(drafts);
  CHECK_ALIGN(u);
  CHECK_ALIGN(temperature);
  CHECK_ALIGN(tokens);
  CHECK_ALIGN(accepted);
  CHECK_ALIGN(logprobs_opt);
  CHECK_ALIGN(ws);
  const long long most = 1ll << 40;
  CHECK(row_stride >= V && row_stride < most, "row_stride=%lld must be at least V=%d", row_stride, V);
  CHECK(user_stride >= V && user_stride < most, "user_stride=%lld must be at least V=%d", user_stride, V);
  if (draft_logits && k > 0) {
    CHECK(draft_row_stride >= V && draft_row_stride < most, "draft_row_stride=%lld must be at least V=%d", draft_row_stride, V);
    CHECK(draft_user_stride >= V && draft_user_stride < most, "draft_user_stride=%lld must be at least V=%d", draft_user_stride, V);
  }
  int st = check_ws(ws, ws_bytes, draft_verify_bytes(b, k, V));
  if (st != Q4_OK) return st;
  DEVICE_OR_RETURN(dev);
  return launch_draft_verify({logits, k > 0 ? draft_logits : nullptr, user_stride, row_stride, draft_user_stride, draft_row_stride,
                              dtype, b, k, V, drafts, u, temperature, tokens, accepted, logprobs_opt},
                             ws, dev, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
