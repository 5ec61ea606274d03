// Attention of few query rows per KV head over an int8 paged cache: what the kernel of
// q4w_attn_decode.cuh is instantiated for, and when.
#include "q4w_attn_decode.cuh"

namespace q4w {
namespace dec {

// The largest NT: O takes NT D / 4 registers, so 128 of them (at head size 64, where 64 rows would still fit,
// four is the most that is built).  This kernel and the tile kernel at the most rows, one KV head, fp16 (bf16),
// us, 64 users of 593000 keys in all: 24 heads of 64 71 and 150 (63, 134), 24 of 128 96 and 195 (89, 148), 16 of
// 256 99 and 207 (93, 174), 8 of 512 122 and 676; 8 users of 19000 keys: 16.6 and 22.5, 25.3 and 25.1 (25.8,
// 24.1), 23 and 28, 24 and 47.
constexpr int max_nt_q8(int D) { return D == 512 ? 1 : D == 256 ? 2 : 4; }

template <typename T>
static int launch_q8(Params& p, int D, int nt, const DeviceInfo& dev, cudaStream_t s) {
  switch (D) {
    case 64: return nt == 1 ? launch<T, 64, 1, true>(p, dev, s) : nt == 2 ? launch<T, 64, 2, true>(p, dev, s) : launch<T, 64, 4, true>(p, dev, s);
    case 128: return nt == 1 ? launch<T, 128, 1, true>(p, dev, s) : nt == 2 ? launch<T, 128, 2, true>(p, dev, s) : launch<T, 128, 4, true>(p, dev, s);
    case 256: return nt == 1 ? launch<T, 256, 1, true>(p, dev, s) : launch<T, 256, 2, true>(p, dev, s);
    default: return launch<T, 512, 1, true>(p, dev, s);
  }
}

}  // namespace dec

bool attn_decode_q8_fits(long long max_rows, int D) { return max_rows <= 8 * dec::max_nt_q8(D); }

size_t attn_decode_q8_ws_bytes(int max_rows, int D, const DeviceInfo& dev) {
  return attn_split_bytes(dev.sms, 8 * dec::nt_of(max_rows), D);
}

int launch_attn_decode_q8(const AttnParams& a, const q4_kv_cache& c, void* ws, const DeviceInfo& dev, cudaStream_t s) {
  dec::Params p = {};
  p.a = a;
  p.group = a.n_q / c.n_kv;
  const int nt = dec::nt_of(a.max_q * p.group);
  p.grid = dev.sms;
  p.split = attn_split(ws, p.grid, 8 * nt, c.head_dim);
  return c.dtype == Q4_BF16 ? dec::launch_q8<__nv_bfloat16>(p, c.head_dim, nt, dev, s)
                            : dec::launch_q8<__half>(p, c.head_dim, nt, dev, s);
}

}  // namespace q4w
