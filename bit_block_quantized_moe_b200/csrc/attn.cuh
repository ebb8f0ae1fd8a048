// Shared by the attention kernels: what they know of a batch, and small device helpers.
#pragma once

#include <cuda.h>
#include <limits.h>

#include "attn_index.h"
#include "kernels.cuh"

namespace moe {

struct KvArgs {
  const int32_t *q_start, *kv_len, *table;
  int n_seqs, max_pages, n_pages;
  int per;     // rows a sequence when q_start is null
  int cap;     // max_pages * page_size
  int log_ps;  // log2(page_size)
};

cudaError_t launch_qk_norm_rope(const moe_attn_dims &d, const uint16_t *qkv, int64_t ld, const float *gq,
                                const float *gk, float eps, const moe_rope *rope, const moe_kv_cache &c,
                                const KvArgs &kv, int T, uint16_t *q_out, uint32_t *status, cudaStream_t s);

constexpr int kAttnSms = 148;               // a window call has one or two CTAs a SM
constexpr int kAttnShares = 2 * kAttnSms;   // the most shares into which its key tiles are cut, one a CTA

struct AttnArgs {
  const uint16_t *q;
  int64_t ld_q;
  const uint16_t *k, *v;
  KvArgs kv;
  int H, V, G, T;
  float scale_log2;  // scale * log2(e)
  int window, n_sinks;
  uint16_t *out;
  uint32_t *status;
  float *part;        // workspace: parts of split groups
  uint32_t *counts;   // workspace header: parts that have come, zero between calls [kAttnShares]
};

// One side of the cache as rows of D elements, boxes of a page's rows (at most `tile`) x 64 elements, 128-byte
// swizzle.
bool make_pages_map(CUtensorMap *map, const uint16_t *cache, int n_pages, const AttnArgs &a, int D, int tile);
size_t attn_part_bytes(const moe_attn_dims &d, int n_seqs, int T);
cudaError_t launch_attn_tc(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s);
cudaError_t launch_attn(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (a0, a1) += (b0, b1) * (c0, c1), (a0, a1) *= (b0, b1), (a0, a1) += (b0, b1): one instruction for both, each lane rounded by itself.
__device__ __forceinline__ void fma2(float &a0, float &a1, float b0, float b1, float c0, float c1) {
  uint64_t acc, b, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(b), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(acc));
}
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
  uint64_t acc, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(acc));
}

__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1) {
  uint64_t acc, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(acc));
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// The sequence of row t, by a whole warp: the number of ends at or before t when the starts do not decrease (the
// caller checks that t lies in that sequence), -1 past the last.
__device__ __forceinline__ int seq_of_row(const KvArgs &kv, int t, int lane) {
  if (!kv.q_start) return t / kv.per;
  int c = 0;
  for (int b = lane; b < kv.n_seqs; b += 32) c += __ldg(kv.q_start + b + 1) <= t;
  c = __reduce_add_sync(0xffffffffu, c);
  return c < kv.n_seqs ? c : -1;
}

// One CTA's threads look the sequences over and report what is out of range.
__device__ __forceinline__ void check_sequences(const KvArgs &kv, int T, uint32_t *status) {
  bool bad = false;
  for (int b = threadIdx.x; b < kv.n_seqs; b += blockDim.x)
    bad |= seq_view(kv.q_start, kv.kv_len, b, kv.per, T, kv.cap).bad;
  if (bad) set_status(status, kStatusBadIndex);
}
#endif

}  // namespace moe
