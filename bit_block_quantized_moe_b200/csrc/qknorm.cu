// Per-head norms of queries and keys with the rotation, in one pass over the projections; keys and values go to
// their rows of the paged cache.
//
// For a head row h of D elements: n = h / sqrt(mean(h^2) + eps) * gain, then for i < r/2 the pair (n_i, n_{i+r/2})
// is turned by position * turn[i].  The angle is kept in turns as a 64-bit fixed-point fraction: position * turn[i]
// mod 2^64 loses whole turns and nothing else, so that the angle of position 2^30 is as exact as that of position 1
// (an fp32 product position * frequency would be off by 0.03 radians at position 500,000).
//
// Bound: HBM (every element read once and written once).  A CTA takes kTok tokens: first its threads make the
// tokens' sines and cosines (r/2 a token) in shared memory, then groups of D/8 lanes take a head row each, 16 bytes
// a lane; the mean is a butterfly over the group, and a pair's partner is r/16 lanes away.
#include <algorithm>

#include "attn.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kTok = 4;  // tokens a CTA

struct NormArgs {
  const uint16_t *qkv;
  int64_t ld;
  const float *gq, *gk;
  float eps;
  int half;  // rotary_dim / 2, 0 without a rotation
  uint16_t *q_out, *k, *v;
  KvArgs kv;
  int H, V, T;
  uint32_t *status;
};

template <int D>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(const __grid_constant__ NormArgs a,
                                                                    const __grid_constant__ moe_rope rope) {
  constexpr int kGroup = D / 8;                  // lanes a head row
  constexpr int kRows = kNormThreads / kGroup;   // head rows a pass of the CTA
  __shared__ float2 cs[kTok][64];
  __shared__ int pos_s[kTok];
  __shared__ int64_t row_s[kTok];
  const int t0 = blockIdx.x * kTok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
  if (warp < kTok) {
    const int t = t0 + warp;
    int pos = INT_MIN;  // no sequence's row
    int64_t row = -1;
    if (t < a.T) {
      const int b = seq_of_row(a.kv, t, lane);
      if (b >= 0) {
        const SeqView s = seq_view(a.kv.q_start, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
        if (t >= s.q0 && t < s.q0 + s.m) {
          pos = s.n - s.m + (t - s.q0);
          if (pos >= 0) {
            row = cache_row(a.kv.table + (size_t)b * a.kv.max_pages, pos, a.kv.log_ps, a.kv.n_pages, a.V);
            if (row < 0 && lane == 0) set_status(a.status, kStatusBadIndex);
          }
        }
      }
    }
    if (lane == 0) {
      pos_s[warp] = pos;
      row_s[warp] = row;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kTok * a.half; i += kNormThreads) {
    const int t = i / a.half, e = i - t * a.half;
    const int pos = pos_s[t];
    if (pos >= 0) {
      const int64_t turns = (int64_t)((uint64_t)pos * rope.turn[e]);  // signed: half a turn each way
      // 2^-63 of the signed fraction is the angle in half turns, which sincospi takes exactly
      float s, c;
      sincospif((float)((double)turns * 0x1p-63), &s, &c);
      cs[t][e] = make_float2(c, s);
    }
  }
  __syncthreads();

  const int heads = a.H + 2 * a.V;
  const int sub = threadIdx.x % kGroup;
  const int e0 = sub * 8;               // this lane's elements
  const int part = a.half / 8;          // lanes to a pair's partner
  const bool turned = e0 < 2 * a.half, upper = e0 >= a.half;
  const int freq0 = upper ? e0 - a.half : e0;
  const int total = kTok * heads;
  const int rounds = (total + kRows - 1) / kRows;
  for (int it = 0; it < rounds; ++it) {
    const int rr = it * kRows + threadIdx.x / kGroup;
    const int tt = rr / heads, h = rr - tt * heads;
    const int t = t0 + tt;
    const int pos = rr < total ? pos_s[tt] : INT_MIN;
    const bool live = rr < total && t < a.T && pos != INT_MIN;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = ldg_nc_v4(a.qkv + (size_t)t * a.ld + (size_t)h * D + e0);
    float x[8];
    unpack8(raw, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
    const float *gain = h < a.H ? a.gq : a.gk;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (gain ? __ldg(gain + e0 + i) : 1.0f);
    if (a.half) {
      // every lane takes part in the exchange; those beyond the rotated part read a lane of their own group
      const int from = turned ? (upper ? lane - part : lane + part) : lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], from);
        if (live && turned && pos >= 0) {
          const float2 w = cs[tt][freq0 + i];
          x[i] = upper ? fmaf(x[i], w.x, y * w.y) : fmaf(x[i], w.x, -(y * w.y));
        }
      }
    }
    if (!live) continue;
    if (h < a.H) {
      uint4 o = pack8(x);
      if (pos < 0) o = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(a.q_out + ((size_t)t * a.H + h) * D + e0) = o;
    } else if (row_s[tt] >= 0) {
      const bool is_k = h < a.H + a.V;
      const int hv = is_k ? h - a.H : h - a.H - a.V;
      uint16_t *dst = (is_k ? a.k : a.v) + ((size_t)row_s[tt] + ((size_t)hv << a.kv.log_ps)) * D + e0;
      *reinterpret_cast<uint4 *>(dst) = is_k ? pack8(x) : raw;
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const moe_attn_dims &d, const uint16_t *qkv, int64_t ld, const float *gq,
                                const float *gk, float eps, const moe_rope *rope, const moe_kv_cache &c,
                                const KvArgs &kv, int T, uint16_t *q_out, uint32_t *status, cudaStream_t s) {
  NormArgs a{qkv, ld, gq, gk, eps, rope ? rope->rotary_dim / 2 : 0, q_out, c.k, c.v, kv, d.n_heads, d.n_kv_heads, T,
             status};
  moe_rope none{};
  const moe_rope &r = rope ? *rope : none;
  const unsigned grid = (unsigned)((T + kTok - 1) / kTok);
  trace_mark(MOE_KERNEL_QK_NORM, false, s);
  if (d.head_dim == 128)
    qk_norm_rope_kernel<128><<<grid, kNormThreads, 0, s>>>(a, r);
  else
    qk_norm_rope_kernel<64><<<grid, kNormThreads, 0, s>>>(a, r);
  trace_mark(MOE_KERNEL_QK_NORM, true, s);
  return cudaGetLastError();
}

}  // namespace moe
