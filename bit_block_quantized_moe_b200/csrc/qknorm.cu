// Per-head norms of queries and keys with the rotation, in one pass over the projections; keys and values go to
// their rows of the paged cache.
//
// For a head row h of D elements: n = h / sqrt(mean(h^2) + eps) * gain, then for i < r/2 the pair (n_i, n_{i+r/2})
// is turned by position * turn[i].  The angle is kept in turns as a 64-bit fixed-point fraction: position * turn[i]
// mod 2^64 loses whole turns and nothing else, so that the angle of position 2^30 is as exact as that of position 1
// (an fp32 product position * frequency would be off by 0.03 radians at position 500,000).
//
// Bound: HBM (every element read once and written once), and close behind it the instructions.  Persistent CTAs take
// kTok tokens a round.  Groups of D/16 lanes take a head row; a lane has two pieces of 8 elements, both partners of
// its 8 pairs, so that the rotation needs no exchange and the mean a butterfly over few lanes.  All rows of a group
// belong to one token, so that a lane keeps its sines and cosines in registers (made by the CTA's threads in shared
// memory, r/2 a token); kDepth rows of the next step are in flight under the present one's arithmetic.  32768 tokens
// of 20 heads take 73 us (4.6 TB/s, 70% of the copy rate); 151 us with one row in flight and the tables read per row,
// 113 us with five in flight and one piece of 8 elements a lane, whose partner lay in another lane (185 instructions a
// piece).  Three rows in flight, or three CTAs a SM, spill registers: 145 to 170 us.
#include <algorithm>

#include "attn.cuh"
#include "half.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kTok = 8;    // tokens a CTA, a warp's angles each
constexpr int kDepth = 2;  // head rows in flight a lane

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
__global__ void __launch_bounds__(kNormThreads, 2) qk_norm_rope_kernel(const __grid_constant__ NormArgs a,
                                                                       const __grid_constant__ moe_rope rope) {
  constexpr int kGroup = D / 16;                         // lanes a head row
  constexpr int kStep = kNormThreads / kGroup / kTok;    // groups a token
  static_assert(kNormThreads / 32 == kTok, "a warp makes a token's angles");
  __shared__ float2 cs[2][kTok][64];
  __shared__ int pos_s[2][kTok];
  __shared__ int64_t row_s[2][kTok];
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = threadIdx.x / kGroup, sub = threadIdx.x % kGroup;
  const int tt = group / kStep, h0 = group % kStep;
  const int heads = a.H + 2 * a.V, steps = (heads + kDepth * kStep - 1) / (kDepth * kStep);
  // this lane's pieces: elements e0 .. e0 + 7 and e1 .. e1 + 7, partners where they are turned
  const bool turned = sub * 8 < a.half;
  const int e0 = turned ? sub * 8 : sub * 16, e1 = turned ? a.half + sub * 8 : sub * 16 + 8;
  auto fetch = [&](int t0, int step, uint4 (&r)[kDepth][2]) {
    const int t = t0 + tt;
    const uint16_t *src = a.qkv + (size_t)min(t, a.T - 1) * a.ld;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int h = h0 + (step * kDepth + i) * kStep;
      const bool in = t < a.T && h < heads;
      r[i][0] = in ? ldg_nc_v4(src + (size_t)h * D + e0) : make_uint4(0, 0, 0, 0);
      r[i][1] = in ? ldg_nc_v4(src + (size_t)h * D + e1) : make_uint4(0, 0, 0, 0);
    }
  };
  // a token's position, cache row and angles, by a warp, two angles a lane
  const uint64_t turn0 = rope.turn[lane], turn1 = rope.turn[lane + 32];
  auto tables = [&](int t0, int par) {
    const int tw = t0 + warp;
    int pos = INT_MIN;  // no sequence's row
    int64_t row = -1;
    if (tw < a.T) {
      const int b = seq_of_row(a.kv, tw, lane);
      if (b >= 0) {
        const SeqView s = seq_view(a.kv.q_start, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
        if (tw >= s.q0 && tw < s.q0 + s.m) {
          pos = s.n - s.m + (tw - s.q0);
          if (pos >= 0) {
            row = cache_row(a.kv.table + (size_t)b * a.kv.max_pages, pos, a.kv.log_ps, a.kv.n_pages, a.V);
            if (row < 0 && lane == 0) set_status(a.status, kStatusBadIndex);
          }
        }
      }
    }
    if (lane == 0) {
      pos_s[par][warp] = pos;
      row_s[par][warp] = row;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (lane + 32 * e >= a.half) break;
      const int64_t turns = (int64_t)((uint64_t)max(pos, 0) * (e ? turn1 : turn0));  // signed: half a turn each way
      // the angle within half a turn: there the fast sine and cosine are good to 2^-20, far below bf16's step
      float sn, cn;
      __sincosf((float)turns * (0x1p-63f * 3.14159265358979f), &sn, &cn);
      cs[par][warp][lane + 32 * e] = make_float2(cn, sn);
    }
  };
  pdl_wait();
  float gq[16], gk[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int e = k < 8 ? e0 + k : e1 + k - 8;
    gq[k] = a.gq ? __ldg(a.gq + e) : 1.f;
    gk[k] = a.gk ? __ldg(a.gk + e) : 1.f;
  }
  uint4 raw[kDepth][2];
  int t0 = blockIdx.x * kTok, par = 0;
  fetch(t0, 0, raw);
  tables(t0, 0);
  for (; t0 < a.T; t0 += gridDim.x * kTok, par ^= 1) {
    // the tables of two rounds stand by turns: one meeting a round, the next round's made before it
    __syncthreads();
    tables(t0 + gridDim.x * kTok, par ^ 1);
    const int t = t0 + tt, pos = pos_s[par][tt];
    const int64_t row = row_s[par][tt];
    const bool live = t < a.T && pos != INT_MIN;
    float cn[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 w = turned ? cs[par][tt][e0 + i] : make_float2(1.f, 0.f);
      cn[i] = w.x;
      sn[i] = w.y;
    }
    for (int step = 0; step < steps; ++step) {
      uint4 next[kDepth][2];
      if (step + 1 < steps)
        fetch(t0, step + 1, next);
      else
        fetch(t0 + gridDim.x * kTok, 0, next);
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        const int h = h0 + (step * kDepth + i) * kStep;
        if ((step * kDepth + i) * kStep >= heads) break;  // no group of the token has a row left
        if (h >= a.H + a.V) {  // a value head: as it is
          if (live && h < heads && row >= 0) {
            uint16_t *dst = a.v + ((size_t)row + ((size_t)(h - a.H - a.V) << a.kv.log_ps)) * D;
            *reinterpret_cast<uint4 *>(dst + e0) = raw[i][0];
            *reinterpret_cast<uint4 *>(dst + e1) = raw[i][1];
          }
          continue;
        }
        float x[8], y[8];
        unpack8(raw[i][0], x);
        unpack8(raw[i][1], y);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) fma2(s0, s1, x[k], y[k], x[k], y[k]);
        float ss = s0 + s1;
        const uint32_t lanes = ((1u << kGroup) - 1u) << (lane & ~(kGroup - 1));  // this group's: its rows are of one kind
#pragma unroll
        for (int o = kGroup / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);  // within 2 units of the last place: far below bf16's step
        const bool is_q = h < a.H;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mul2(x[k], y[k], inv, inv);
          mul2(x[k], y[k], is_q ? gq[k] : gk[k], is_q ? gq[k + 8] : gk[k + 8]);
        }
        if (turned) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // (x, y) (c, c) + (-y, x) (s, s)
            float u = -y[k] * sn[k], v = x[k] * sn[k];
            fma2(u, v, x[k], y[k], cn[k], cn[k]);
            x[k] = u;
            y[k] = v;
          }
        }
        if (!live) continue;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if (is_q) {
          uint16_t *dst = a.q_out + ((size_t)t * a.H + h) * D;
          *reinterpret_cast<uint4 *>(dst + e0) = pos < 0 ? zero : pack8(x);
          *reinterpret_cast<uint4 *>(dst + e1) = pos < 0 ? zero : pack8(y);
        } else if (row >= 0) {
          uint16_t *dst = a.k + ((size_t)row + ((size_t)(h - a.H) << a.kv.log_ps)) * D;
          *reinterpret_cast<uint4 *>(dst + e0) = pack8(x);
          *reinterpret_cast<uint4 *>(dst + e1) = pack8(y);
        }
      }
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        raw[i][0] = next[i][0];
        raw[i][1] = next[i][1];
      }
    }
  }
  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const moe_attn_dims &d, const uint16_t *qkv, int64_t ld, const float *gq,
                                const float *gk, float eps, const moe_rope *rope, const moe_kv_cache &c,
                                const KvArgs &kv, int T, uint16_t *q_out, uint32_t *status, cudaStream_t s) {
  NormArgs a{qkv, ld, gq, gk, eps, rope ? rope->rotary_dim / 2 : 0, q_out, c.k, c.v, kv, d.n_heads, d.n_kv_heads, T,
             status};
  moe_rope none{};
  const moe_rope &r = rope ? *rope : none;
  const unsigned grid = (unsigned)std::min((T + kTok - 1) / kTok, 2 * 148);  // two CTAs a SM
  trace_mark(MOE_KERNEL_QK_NORM, false, s);
  const cudaError_t err = d.head_dim == 128 ? launch_dependent(qk_norm_rope_kernel<128>, grid, kNormThreads, 0, 1, s, a, r)
                                            : launch_dependent(qk_norm_rope_kernel<64>, grid, kNormThreads, 0, 1, s, a, r);
  trace_mark(MOE_KERNEL_QK_NORM, true, s);
  return err;
}

}  // namespace moe
