// C ABI entry points of the attention half: argument checks, workspace layout, launches.
#include <math.h>

#include "attn.cuh"

namespace moe {

static bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

static bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

static moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr size_t kWsHeader = 2048;  // the sticky status word; from byte 256 on the counts of parts
constexpr size_t kWsCounts = 256;
static_assert(kWsCounts + kAttnShares * 4 <= kWsHeader, "the counts lie in the header");

constexpr int32_t kMaxRows = 1 << 30;  // so that a row's number and a grid's step beyond it stay below 2^31

static bool linear_dims_ok(int32_t T, int32_t K, int32_t N) {
  return T >= 0 && T <= kMaxRows && K >= 8 && K <= 65536 && K % 8 == 0 && N >= 1 && N <= 262144;
}

static bool attn_dims_ok(const moe_attn_dims *d) {
  if (!d) return false;
  if (d->head_dim != 64 && d->head_dim != 128) return false;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return false;
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads > 1024 || d->n_heads % d->n_kv_heads) return false;
  return d->n_heads / d->n_kv_heads <= 128;
}

// The batch and the cache of a call with T > 0 rows.
static moe_status check_batch(const moe_attn_dims &d, const moe_kv_cache *c, const moe_kv_batch *b, int32_t T,
                              KvArgs *kv) {
  if (!c || !b || !c->k || !c->v || !b->kv_len || !b->page_table) return MOE_ERR_ARG;
  if (c->n_pages < 1 || (int64_t)c->n_pages * d.n_kv_heads * d.page_size > INT32_MAX) return MOE_ERR_ARG;
  if (b->n_seqs < 1 || b->n_seqs > 65536 || b->max_pages < 1) return MOE_ERR_ARG;
  if ((int64_t)b->max_pages * d.page_size > (1 << 30)) return MOE_ERR_ARG;
  if (!b->q_start && T % b->n_seqs) return MOE_ERR_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_ALIGN;
  kv->q_start = b->q_start;
  kv->kv_len = b->kv_len;
  kv->table = b->page_table;
  kv->n_seqs = b->n_seqs;
  kv->max_pages = b->max_pages;
  kv->n_pages = c->n_pages;
  kv->per = b->q_start ? 0 : T / b->n_seqs;
  kv->cap = b->max_pages * d.page_size;
  kv->log_ps = d.page_size == 16 ? 4 : d.page_size == 32 ? 5 : d.page_size == 64 ? 6 : 7;
  return MOE_OK;
}

static size_t cache_bytes(const moe_attn_dims &d, const moe_kv_cache &c) {
  return (size_t)c.n_pages * d.n_kv_heads * d.page_size * d.head_dim * 2;
}

// Bytes of T rows of `width` elements, ld apart.
static size_t rows_bytes(int32_t T, int64_t ld, int64_t width) { return ((size_t)(T - 1) * ld + width) * 2; }

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_bytes(int32_t max_T, int32_t K, int32_t N) {
  if (!linear_dims_ok(max_T, K, N)) return 0;
  return kWsHeader;
}

moe_status moe_linear(const uint16_t *x, int64_t ld_x, const uint16_t *w, const float *bias, moe_act act,
                      const float *resid, void *out, int32_t T, int32_t K, int32_t N, void *workspace,
                      size_t ws_bytes, moe_stream_t stream) {
  if (!linear_dims_ok(T, K, N)) return MOE_ERR_ARG;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out || !workspace) return MOE_ERR_ARG;
  if (ld_x < K || ld_x % 8 || ld_x > (1ll << 31)) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out) || !aligned16(workspace) || !aligned16(bias) ||
      !aligned16(resid))
    return MOE_ERR_ALIGN;
  const size_t ob = (size_t)T * N * (resid ? 4 : 2);
  if (overlaps(out, ob, x, rows_bytes(T, ld_x, K)) || overlaps(out, ob, w, (size_t)N * K * 2)) return MOE_ERR_ARG;
  if (bias && overlaps(out, ob, bias, (size_t)N * 4)) return MOE_ERR_ARG;
  if (resid && static_cast<const void *>(resid) != out && overlaps(out, ob, resid, ob)) return MOE_ERR_ARG;
  if (ws_bytes < moe_linear_workspace_bytes(T, K, N)) return MOE_ERR_WORKSPACE;
  const moe_status dev = device_ok();
  if (dev != MOE_OK) return dev;
  return cuda_status(launch_linear(x, ld_x, w, bias, act, resid, out, T, K, N, static_cast<uint32_t *>(workspace),
                                   reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_rope_init(double theta, int32_t rotary_dim, moe_rope *rope) {
  if (!rope || !(theta >= 1.0) || !(theta <= 1e30) || rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16)
    return MOE_ERR_ARG;
  rope->rotary_dim = rotary_dim;
  rope->reserved = 0;
  for (int i = 0; i < 64; ++i) rope->turn[i] = 0;
  // theta^(-2i/r) radians a position, over 2 pi, in units of 2^-64: a 64-bit long double keeps every bit
  const long double pi2 = 6.283185307179586476925286766559005768L;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const long double f = powl((long double)theta, -2.0L * i / rotary_dim) / pi2;  // at most 0.16
    rope->turn[i] = (uint64_t)ldexpl(f, 64);
  }
  return MOE_OK;
}

size_t moe_attn_workspace_bytes(const moe_attn_dims *dims, int32_t n_seqs, int32_t max_T) {
  if (!attn_dims_ok(dims) || n_seqs < 1 || n_seqs > 65536 || max_T < 0 || max_T > kMaxRows) return 0;
  return kWsHeader + attn_part_bytes(*dims, n_seqs, max_T);
}

moe_status moe_qk_norm_rope(const moe_attn_dims *dims, const uint16_t *qkv, int64_t ld_qkv, const float *q_gain,
                            const float *k_gain, float eps, const moe_rope *rope, const moe_kv_cache *cache,
                            const moe_kv_batch *batch, int32_t T, uint16_t *q_out, void *workspace, size_t ws_bytes,
                            moe_stream_t stream) {
  if (!attn_dims_ok(dims) || T < 0 || T > kMaxRows || !(eps >= 0.f)) return MOE_ERR_ARG;
  if (rope && (rope->rotary_dim < 16 || rope->rotary_dim > dims->head_dim || rope->rotary_dim % 16)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!qkv || !q_out || !workspace) return MOE_ERR_ARG;
  KvArgs kv;
  const moe_status st = check_batch(*dims, cache, batch, T, &kv);
  if (st != MOE_OK) return st;
  const int64_t width = (int64_t)(dims->n_heads + 2 * dims->n_kv_heads) * dims->head_dim;
  if (ld_qkv < width || ld_qkv % 8 || ld_qkv > (1ll << 31)) return MOE_ERR_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(workspace) || !aligned16(q_gain) || !aligned16(k_gain))
    return MOE_ERR_ALIGN;
  const size_t qb = rows_bytes(T, ld_qkv, width), ob = (size_t)T * dims->n_heads * dims->head_dim * 2;
  const size_t cb = cache_bytes(*dims, *cache);
  if (overlaps(q_out, ob, qkv, qb) || overlaps(cache->k, cb, qkv, qb) || overlaps(cache->v, cb, qkv, qb) ||
      overlaps(q_out, ob, cache->k, cb) || overlaps(q_out, ob, cache->v, cb) || overlaps(cache->k, cb, cache->v, cb))
    return MOE_ERR_ARG;
  if (ws_bytes < moe_attn_workspace_bytes(dims, batch->n_seqs, T)) return MOE_ERR_WORKSPACE;
  const moe_status dev = device_ok();
  if (dev != MOE_OK) return dev;
  return cuda_status(launch_qk_norm_rope(*dims, qkv, ld_qkv, q_gain, k_gain, eps, rope, *cache, kv, T, q_out,
                                         static_cast<uint32_t *>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_attn_forward(const moe_attn_dims *dims, const uint16_t *q, int64_t ld_q, const moe_kv_cache *cache,
                            const moe_kv_batch *batch, int32_t T, float scale, int32_t window, int32_t n_sinks,
                            uint16_t *out, void *workspace, size_t ws_bytes, moe_stream_t stream) {
  if (!attn_dims_ok(dims) || T < 0 || T > kMaxRows || window < 0 || n_sinks < 0) return MOE_ERR_ARG;
  if (!isfinite(scale * 1.4426950408889634f)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !out || !workspace) return MOE_ERR_ARG;
  AttnArgs a{};
  const moe_status st = check_batch(*dims, cache, batch, T, &a.kv);
  if (st != MOE_OK) return st;
  const int64_t width = (int64_t)dims->n_heads * dims->head_dim;
  if (ld_q < width || ld_q % 8 || ld_q > (1ll << 31)) return MOE_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return MOE_ERR_ALIGN;
  const size_t ob = (size_t)T * width * 2, cb = cache_bytes(*dims, *cache);
  if (overlaps(out, ob, q, rows_bytes(T, ld_q, width)) || overlaps(out, ob, cache->k, cb) ||
      overlaps(out, ob, cache->v, cb))
    return MOE_ERR_ARG;
  if (ws_bytes < moe_attn_workspace_bytes(dims, batch->n_seqs, T)) return MOE_ERR_WORKSPACE;
  const moe_status dev = device_ok();
  if (dev != MOE_OK) return dev;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.q = q;
  a.ld_q = ld_q;
  a.k = cache->k;
  a.v = cache->v;
  a.H = dims->n_heads;
  a.V = dims->n_kv_heads;
  a.G = a.H / a.V;
  a.T = T;
  // scale 0 weighs all seen keys alike, as this does, and keeps masked scores at -inf
  a.scale_log2 = scale * 1.4426950408889634f;
  if (a.scale_log2 == 0.f) a.scale_log2 = 1e-37f;
  // positions stay below 2^30
  a.window = window < (1 << 30) ? window : 1 << 30;
  a.n_sinks = n_sinks < (1 << 30) ? n_sinks : 1 << 30;
  a.out = out;
  a.status = reinterpret_cast<uint32_t *>(ws);
  a.counts = reinterpret_cast<uint32_t *>(ws + kWsCounts);
  a.part = reinterpret_cast<float *>(ws + kWsHeader);
  return cuda_status(launch_attn(*dims, a, *cache, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
