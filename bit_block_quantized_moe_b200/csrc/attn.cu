// Attention of verify windows (1 to 8 new tokens a sequence) over the paged cache, on the legacy tensor path
// (mma.sync): the work is reading the cache once, and a window's few rows fill 16-row products, not 128-row ones.
//
// The query heads of a group share their key/value head, so that a tile's rows are (token, head of the group) pairs:
// row r is token r / G, head r % G.  One pass over the keys with the running maximum and sum of the softmax:
//   s_j = scale q.k_j,  m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),  o' = o e^(m - m') + ...
// in base 2 with scale * log2(e) folded in.
//
// Split: all 128-key tiles of all (sequence, key/value head, row tile) groups stand in one line, which is cut into
// equal shares, one a CTA, whatever the lengths (they are read on the device, so that a captured graph follows them).
// A CTA's share is one stream of loads through its ring of stages, across group ends.  A group that is cut leaves
// parts (m, l, o) in the workspace; the CTA that brings the last one joins them in share order, so that the result
// does not depend on which that is.
//   last warp        : TMA of K and V, a page at a time, into the ring; 128-byte swizzle;
//   WM x WK warps    : 16 rows and 1/WK of a tile's keys each, with m, l, o of their own, no waits on one another
//                      but at a group's end, where they join pairwise.
// Rows of V that no query of the window sees are masked in the registers that feed the product, so that nothing behind
// them can reach an output.  Every wait is bounded (sync.cuh).
#include <algorithm>

#include "attn.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;        // keys a tile
constexpr int kLogBK = 7;

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
template <int D, int WM, int WK>
struct WinCfg {
  static constexpr int kWarps = WM * WK;            // beside the producer
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kRows = 16 * WM;
  static constexpr int kKeys = kBK / WK;            // keys a warp
  static constexpr int kTileBytes = kBK * D * 2;    // K or V of a stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kOut = D / 2;                // accumulators a lane
  static constexpr int kJoinBytes = WM * (WK / 2) * 32 * (kOut + 4) * 4;
  static constexpr int kHalfBytes = kBK * 128;      // 64 columns of a tile, one swizzle row a key
  static constexpr int kSmem = kStages * kStageBytes + kJoinBytes;
};

template <int STAGES>
struct WinBars {
  uint64_t full[STAGES], empty[STAGES];
  int partial[STAGES];       // some row does not see some key of the tile
  uint32_t bad[STAGES][4];   // keys whose page is outside the cache
  int abort;
};

struct WinArgs {
  AttnArgs a;
  int row_tiles;
};

// Where a CTA stands in the line of tiles: tile t of group g (key/value head and row tile) of sequence b.
struct Cursor {
  int b, g, t, nt;
  SeqView s;
  TileRange r;

  __device__ __forceinline__ void sequence(const AttnArgs &a, int seq) {
    b = seq;
    s = seq_view(nullptr, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
    r = tile_range(s.n - s.m, s.n - 1, s.n, a.window, a.n_sinks, kLogBK);
    nt = max(r.count, 1);  // an empty sequence has one tile in which nothing is seen
  }
  __device__ __forceinline__ void advance(const AttnArgs &a, int groups) {
    if (++t < nt) return;
    t = 0;
    if (++g < groups) return;
    g = 0;
    if (b + 1 < a.kv.n_seqs) sequence(a, b + 1);
  }
  __device__ __forceinline__ int key0() const { return tile_of(r, t) << kLogBK; }
};

template <class Bars>
__device__ __forceinline__ bool win_wait(uint64_t *bar, uint32_t parity, Bars &B, uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int *>(&B.abort)) return false;
  if (!mbar_wait(bar, parity)) {
    set_status(status, kStatusTimeout);
    B.abort = 1;
    return false;
  }
  return true;
}

// Whether 16 bytes hold a bf16 infinity or NaN.
__device__ __forceinline__ bool not_finite8(const uint4 &x) {
  const uint32_t e[4] = {x.x, x.y, x.z, x.w};
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) bad |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

template <int D, int WM, int WK>
__global__ void __launch_bounds__(WinCfg<D, WM, WK>::kThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ WinArgs w) {
  using C = WinCfg<D, WM, WK>;
  extern __shared__ __align__(1024) uint8_t win_smem[];
  __shared__ WinBars<C::kStages> B;
  __shared__ long long scan_s[C::kThreads / 32];
  __shared__ int found_b, last_s;
  __shared__ long long found_base;
  const AttnArgs &a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int wm = warp % WM, wk = warp / WM;
  const int groups = a.V * w.row_tiles, rows = a.kv.per * a.G;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], C::kWarps);
    }
    B.abort = 0;
    mbar_fence_init();
  }

  // ---- this CTA's share [x0, x1) of the line, and the sequence in which it begins
  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
  long long total = 0;
  for (int c0 = 0; c0 < a.kv.n_seqs; c0 += C::kThreads) {
    const int b = c0 + threadIdx.x;
    Cursor q;
    q.nt = 0;
    if (b < a.kv.n_seqs) q.sequence(a, b);
    total += q.nt;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) scan_s[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < C::kThreads / 32; ++i) total += scan_s[i];
  total *= groups;
  const int shares = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= shares) return;
  const long long x0 = total * blockIdx.x / shares, x1 = total * (blockIdx.x + 1) / shares;
  long long base = 0;
  for (int c0 = 0; c0 < a.kv.n_seqs && base <= x0; c0 += C::kThreads) {
    const int b = c0 + threadIdx.x;
    Cursor q;
    q.nt = 0;
    if (b < a.kv.n_seqs) q.sequence(a, b);
    long long incl = q.nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) scan_s[warp] = incl;
    __syncthreads();
    long long before = incl - q.nt, sum = 0;
#pragma unroll
    for (int i = 0; i < C::kThreads / 32; ++i) {
      if (i < warp) before += scan_s[i];
      sum += scan_s[i];
    }
    const long long at = base + before * groups;
    if (q.nt > 0 && at <= x0 && x0 < at + (long long)q.nt * groups) {
      found_b = b;
      found_base = at;
    }
    base += sum * groups;
  }
  __syncthreads();
  Cursor cur;
  cur.sequence(a, found_b);
  cur.g = (int)((x0 - found_base) / cur.nt);
  cur.t = (int)((x0 - found_base) % cur.nt);

  if (warp == C::kWarps) {
    // ---- producer: lane l < pages has page l of a tile ----
    const int ps = 1 << a.kv.log_ps, pages = kBK >> a.kv.log_ps;
    int st = 0;
    uint32_t ph = 1;
    long long issued = 0;
    for (long long x = x0; x < x1; ++x) {
      const int j0 = cur.key0(), n = cur.s.n, p0 = n - cur.s.m, hv = cur.g / w.row_tiles;
      const int a0 = j0 + (lane << a.kv.log_ps), e0 = a0 + ps;
      const bool seen = lane < pages && a0 < n && (a.window <= 0 || e0 - 1 > p0 - a.window || a0 < a.n_sinks);
      const int page = seen ? __ldg(a.kv.table + (size_t)cur.b * a.kv.max_pages + (a0 >> a.kv.log_ps)) : 0;
      const bool ok = seen && page >= 0 && page < a.kv.n_pages;
      const uint32_t good = __ballot_sync(0xffffffffu, ok), wrong = __ballot_sync(0xffffffffu, seen && !ok);
      if (!__all_sync(0xffffffffu, win_wait(&B.empty[st], ph, B, a.status))) break;
      if (lane == 0) {
        B.partial[st] = wrong || !tile_full(p0, n - 1, j0, kBK, n, a.window, a.n_sinks);
        B.bad[st][0] = B.bad[st][1] = B.bad[st][2] = B.bad[st][3] = 0;
        if (wrong) {
          for (int k = 0; k < kBK; ++k)
            if (wrong >> (k >> a.kv.log_ps) & 1) B.bad[st][k >> 5] |= 1u << (k & 31);
          set_status(a.status, kStatusBadIndex);
        }
        mbar_arrive_expect_tx(&B.full[st], (uint32_t)(__popc(good) * ps * D * 4));
      }
      __syncwarp();
      if (ok) {
        const int row = (page * a.V + hv) << a.kv.log_ps;  // below 2^31: checked on the host
        uint8_t *dst = win_smem + st * C::kStageBytes + lane * ps * 128;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_2d(dst + h * C::kHalfBytes, &kmap, h * 64, row, &B.full[st]);
          tma_load_2d(dst + C::kTileBytes + h * C::kHalfBytes, &vmap, h * 64, row, &B.full[st]);
        }
      }
      __syncwarp();
      ++issued;
      if (++st == C::kStages) {
        st = 0;
        ph ^= 1;
      }
      cur.advance(a, groups);
    }
    // every copy issued must land before the CTA exits, also after an abort
    for (long long t = issued > C::kStages ? issued - C::kStages : 0; t < issued; ++t)
      if (!mbar_wait(&B.full[t % C::kStages], (uint32_t)(t / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
    return;
  }

  // ---- the other warps ----
  const uint32_t smem0 = smem_u32(win_smem);
  uint32_t phase = 0;
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float ma = 0.f, mb = 0.f, la = 0.f, lb = 0.f;
  int r0 = 0, hv = 0, base_pos = 0, pa = -1, pb = -1, cs = 0;
  bool fresh = true;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      // the queries of this warp's 16 rows, as A fragments
      fresh = false;
      hv = cur.g / w.row_tiles;
      r0 = (cur.g - hv * w.row_tiles) * C::kRows;
      base_pos = cur.s.n - cur.s.m;
      const int ra = r0 + 16 * wm + g, rb = ra + 8;
      pa = ra < rows ? base_pos + ra / a.G : -1;
      pb = rb < rows ? base_pos + rb / a.G : -1;
      const uint16_t *qa = a.q + (size_t)(cur.s.q0 + ra / a.G) * a.ld_q + (size_t)(hv * a.G + ra % a.G) * D;
      const uint16_t *qb = a.q + (size_t)(cur.s.q0 + rb / a.G) * a.ld_q + (size_t)(hv * a.G + rb % a.G) * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][0] = ra < rows ? __ldg(reinterpret_cast<const uint32_t *>(qa + 16 * k + 2 * c)) : 0u;
        qf[k][1] = rb < rows ? __ldg(reinterpret_cast<const uint32_t *>(qb + 16 * k + 2 * c)) : 0u;
        qf[k][2] = ra < rows ? __ldg(reinterpret_cast<const uint32_t *>(qa + 16 * k + 8 + 2 * c)) : 0u;
        qf[k][3] = rb < rows ? __ldg(reinterpret_cast<const uint32_t *>(qb + 16 * k + 8 + 2 * c)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      ma = mb = -INFINITY;
      la = lb = 0.f;
    }
    const int j0 = cur.key0(), n = cur.s.n, k0 = wk * C::kKeys;
    const uint32_t st = smem0 + (uint32_t)cs * C::kStageBytes;
    win_wait(&B.full[cs], phase, B, a.status);
    const bool partial = B.partial[cs];
    // the warp's keys that some row sees and whose values are finite (bit i: key k0 + i), and those seen but not finite
    unsigned long long use = ~0ull, flagged = 0;
    if (partial) {
      use = 0;
#pragma unroll
      for (int h = 0; h < C::kKeys; h += 32) {
        const int kk = k0 + h + (lane & (C::kKeys < 32 ? C::kKeys - 1 : 31)), j = j0 + kk;
        const bool live = j < n && (a.window <= 0 || base_pos - j < a.window || j < a.n_sinks) &&
                          !(B.bad[cs][kk >> 5] >> (kk & 31) & 1);
        bool bad = false;
        // 0 * v is NaN when v is not finite: where rows differ in what they see, such a key is left out of the
        // product, and the rows that see it become NaN
        if (live && a.kv.per > 1) {
          const uint8_t *v = win_smem + cs * C::kStageBytes + C::kTileBytes + kk * 128;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            bad |= not_finite8(*reinterpret_cast<const uint4 *>(v + (i >> 3) * C::kHalfBytes + (((i & 7) + lane) & 7) * 16));
        }
        const unsigned long long lv = __ballot_sync(0xffffffffu, live && !bad), bd = __ballot_sync(0xffffffffu, live && bad);
        use |= lv << h;
        flagged |= bd << h;
      }
    }

    float sc[C::kKeys / 8][4];
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < C::kKeys / 16; ++i) {
      const int r = k0 + 16 * i + (lane & 7) + ((lane & 16) ? 8 : 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int ch = 2 * k + ((lane >> 3) & 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(st + (uint32_t)((ch >> 3) * C::kHalfBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4)), b0, b1, b2, b3);
        mma_bf16_16816(sc[2 * i], qf[k], b0, b1, sc[2 * i]);
        mma_bf16_16816(sc[2 * i + 1], qf[k], b2, b3, sc[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] *= a.scale_log2;
    bool nan_a = false, nan_b = false;
    if (partial) {
#pragma unroll
      for (int i = 0; i < C::kKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = 8 * i + 2 * c + e, j = j0 + k0 + kk;
          const bool in = (use | flagged) >> kk & 1, bad = flagged >> kk & 1;
          const bool va = in && key_seen(pa, j, n, a.window, a.n_sinks), vb = in && key_seen(pb, j, n, a.window, a.n_sinks);
          nan_a |= bad && va;
          nan_b |= bad && vb;
          if (!va) sc[i][e] = -INFINITY;
          if (!vb) sc[i][2 + e] = -INFINITY;
        }
    }
    float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i) {
      xa = fmaxf(xa, fmaxf(sc[i][0], sc[i][1]));
      xb = fmaxf(xb, fmaxf(sc[i][2], sc[i][3]));
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, d));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, d));
    }
    const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
    // nothing seen yet: subtract 0, so that e^(-inf - 0) = 0
    const float sa = na == -INFINITY ? 0.f : na, sb = nb == -INFINITY ? 0.f : nb;
    const float fa = ex2(ma - sa), fb = ex2(mb - sb);
    ma = na;
    mb = nb;
    float ta = nan_a ? NAN : 0.f, tb = nan_b ? NAN : 0.f;
    uint32_t pf[C::kKeys / 8][2];
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i) {
      const float e0 = ex2(sc[i][0] - sa), e1 = ex2(sc[i][1] - sa);
      const float e2 = ex2(sc[i][2] - sb), e3 = ex2(sc[i][3] - sb);
      ta += e0 + e1;
      tb += e2 + e3;
      pf[i][0] = pack_bf16x2(e0, e1);
      pf[i][1] = pack_bf16x2(e2, e3);
    }
    la = la * fa + ta;
    lb = lb * fb + tb;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      o[i][0] *= fa;
      o[i][1] *= fa;
      o[i][2] *= fb;
      o[i][3] *= fb;
    }
#pragma unroll
    for (int i = 0; i < C::kKeys / 16; ++i) {
      const uint32_t af[4] = {pf[2 * i][0], pf[2 * i][1], pf[2 * i + 1][0], pf[2 * i + 1][1]};
      const int r = k0 + 16 * i + (lane & 15);
      // this lane's keys of the two halves of the fragment: 2c, 2c + 1 and 8 more
      const uint32_t u = (uint32_t)(use >> (16 * i + 2 * c));
      const uint32_t v0 = (u & 1 ? 0xffffu : 0u) | (u & 2 ? 0xffff0000u : 0u);
      const uint32_t v1 = (u & 256 ? 0xffffu : 0u) | (u & 512 ? 0xffff0000u : 0u);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const int ch = 2 * d + (lane >> 4);
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(st + (uint32_t)(C::kTileBytes + (ch >> 3) * C::kHalfBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4)), b0,
                  b1, b2, b3);
        if (partial) {
          b0 &= v0;
          b1 &= v1;
          b2 &= v0;
          b3 &= v1;
        }
        mma_bf16_16816(o[2 * d], af, b0, b1, o[2 * d]);
        mma_bf16_16816(o[2 * d + 1], af, b2, b3, o[2 * d + 1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.empty[cs]);
    if (++cs == C::kStages) {
      cs = 0;
      phase ^= 1;
    }

    if (cur.t + 1 == cur.nt || x + 1 == x1) {
      // ---- the end of this CTA's part of the group: join the WK warps of each row tile pairwise
      fresh = true;
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, d);
        lb += __shfl_xor_sync(0xffffffffu, lb, d);
      }
      float *join = reinterpret_cast<float *>(win_smem + C::kStages * C::kStageBytes);
#pragma unroll
      for (int h = WK / 2; h > 0; h >>= 1) {
        if (wk >= h && wk < 2 * h) {
          float *q = join + (size_t)((wk - h) * WM + wm) * 32 * (C::kOut + 4) + lane;
#pragma unroll
          for (int i = 0; i < C::kOut; ++i) q[32 * i] = o[i >> 2][i & 3];
          q[32 * C::kOut] = ma;
          q[32 * (C::kOut + 1)] = mb;
          q[32 * (C::kOut + 2)] = la;
          q[32 * (C::kOut + 3)] = lb;
        }
        named_bar(1, C::kWarps * 32);
        if (wk < h) {
          const float *q = join + (size_t)(wk * WM + wm) * 32 * (C::kOut + 4) + lane;
          const float m2a = q[32 * C::kOut], m2b = q[32 * (C::kOut + 1)];
          const float ja = fmaxf(ma, m2a), jb = fmaxf(mb, m2b);
          const float ua = ja == -INFINITY ? 0.f : ja, ub = jb == -INFINITY ? 0.f : jb;
          const float f0 = ex2(ma - ua), f1 = ex2(m2a - ua), f2 = ex2(mb - ub), f3 = ex2(m2b - ub);
          ma = ja;
          mb = jb;
          la = la * f0 + q[32 * (C::kOut + 2)] * f1;
          lb = lb * f2 + q[32 * (C::kOut + 3)] * f3;
#pragma unroll
          for (int i = 0; i < C::kOut; ++i) {
            const float v = q[32 * i];
            o[i >> 2][i & 3] = (i & 2) ? o[i >> 2][i & 3] * f2 + v * f3 : o[i >> 2][i & 3] * f0 + v * f1;
          }
        }
        named_bar(1, C::kWarps * 32);
      }
      const long long gs = x - cur.t, ge = gs + cur.nt;
      const bool whole = gs >= x0 && ge <= x1;
      const int ra = 16 * wm + g, live = min(rows - r0, C::kRows);
      if (whole) {
        if (wk == 0) {
          const float ia = la == 0.f ? 0.f : 1.0f / la, ib = lb == 0.f ? 0.f : 1.0f / lb;
          const int qa = r0 + ra, qb = qa + 8;
          uint16_t *da = a.out + ((size_t)(cur.s.q0 + qa / a.G) * a.H + (size_t)hv * a.G + qa % a.G) * D + 2 * c;
          uint16_t *db = a.out + ((size_t)(cur.s.q0 + qb / a.G) * a.H + (size_t)hv * a.G + qb % a.G) * D + 2 * c;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            if (ra < live) *reinterpret_cast<uint32_t *>(da + 8 * i) = pack_bf16x2(o[i][0] * ia, o[i][1] * ia);
            if (ra + 8 < live) *reinterpret_cast<uint32_t *>(db + 8 * i) = pack_bf16x2(o[i][2] * ib, o[i][3] * ib);
          }
        }
      } else {
        // parts: slot 0 of a share for the group that it begins with, slot 1 for the one that it ends with
        constexpr size_t kPart = (size_t)C::kRows * (D + 2);
        float *po = a.part + ((size_t)blockIdx.x * 2 + (gs > x0)) * kPart, *pm = po + (size_t)C::kRows * D;
        if (wk == 0) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            if (ra < live) __stcg(reinterpret_cast<float2 *>(po + (size_t)ra * D + 8 * i + 2 * c), make_float2(o[i][0], o[i][1]));
            if (ra + 8 < live)
              __stcg(reinterpret_cast<float2 *>(po + (size_t)(ra + 8) * D + 8 * i + 2 * c), make_float2(o[i][2], o[i][3]));
          }
          if (c == 0) {
            if (ra < live) __stcg(reinterpret_cast<float2 *>(pm + 2 * ra), make_float2(ma, la));
            if (ra + 8 < live) __stcg(reinterpret_cast<float2 *>(pm + 2 * (ra + 8)), make_float2(mb, lb));
          }
          __threadfence();
        }
        // the shares that hold this group; each share is the first of at most one cut group, whose count it keeps
        const int c0 = (int)(((gs + 1) * shares - 1) / total), c1 = (int)((ge * shares - 1) / total);
        named_bar(1, C::kWarps * 32);
        if (threadIdx.x == 0) {
          __threadfence();
          const uint32_t before = atomicAdd(a.counts + c0, 1u);
          last_s = before == (uint32_t)(c1 - c0);
          if (last_s) a.counts[c0] = 0;  // for the next call
          __threadfence();
        }
        named_bar(1, C::kWarps * 32);
        if (last_s) {
          const bool late = gs > total * c0 / shares;  // the first part lies in slot 1
          for (int i = threadIdx.x; i < live * (D / 2); i += C::kWarps * 32) {
            const int r = i / (D / 2), d = 2 * (i % (D / 2));
            float m = -INFINITY, l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 8
            for (int k = c0; k <= c1; ++k) {
              const float *pk = a.part + ((size_t)k * 2 + (k == c0 && late)) * kPart;
              const float2 ml = __ldcg(reinterpret_cast<const float2 *>(pk + (size_t)C::kRows * D + 2 * r));
              const float2 v = __ldcg(reinterpret_cast<const float2 *>(pk + (size_t)r * D + d));
              const float nm = fmaxf(m, ml.x), u = nm == -INFINITY ? 0.f : nm;
              const float f0 = ex2(m - u), f1 = ex2(ml.x - u);
              m = nm;
              l = l * f0 + ml.y * f1;
              y0 = y0 * f0 + v.x * f1;
              y1 = y1 * f0 + v.y * f1;
            }
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            const int rg = r0 + r;
            uint16_t *dst = a.out + ((size_t)(cur.s.q0 + rg / a.G) * a.H + (size_t)hv * a.G + rg % a.G) * D + d;
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(y0 * inv, y1 * inv);
          }
        }
        named_bar(1, C::kWarps * 32);
      }
    }
    cur.advance(a, groups);
  }
}

template <int D, int WM, int WK>
cudaError_t launch(WinArgs w, const moe_kv_cache &c, cudaStream_t s) {
  using C = WinCfg<D, WM, WK>;
  CUtensorMap km, vm;
  if (!make_pages_map(&km, c.k, c.n_pages, w.a, D) || !make_pages_map(&vm, c.v, c.n_pages, w.a, D))
    return cudaErrorInvalidValue;
  w.row_tiles = (w.a.kv.per * w.a.G + C::kRows - 1) / C::kRows;
  cudaError_t err =
      cudaFuncSetAttribute(attn_window_kernel<D, WM, WK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  attn_window_kernel<D, WM, WK><<<kAttnShares, C::kThreads, C::kSmem, s>>>(km, vm, w);
  return cudaGetLastError();
}

// Rows of a window: one, two or four 16-row tiles side by side; more rows than 64 walk the keys again.
template <int D>
cudaError_t launch_d(const WinArgs &w, const moe_kv_cache &c, cudaStream_t s) {
  const int rows = w.a.kv.per * w.a.G;
  if (rows <= 16) return launch<D, 1, 8>(w, c, s);
  if (rows <= 32) return launch<D, 2, 4>(w, c, s);
  return launch<D, 4, 2>(w, c, s);
}

}  // namespace

bool make_pages_map(CUtensorMap *map, const uint16_t *cache, int n_pages, const AttnArgs &a, int D) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)n_pages * a.V << a.kv.log_ps};  // rows below 2^31
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, 1u << a.kv.log_ps};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(cache), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t attn_part_bytes(const moe_attn_dims &d, int, int) { return (size_t)kAttnShares * 2 * 64 * (d.head_dim + 2) * 4; }

cudaError_t launch_attn(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s) {
  WinArgs w{a, 1};
  trace_mark(MOE_KERNEL_ATTN, false, s);
  const bool window = !a.kv.q_start && a.kv.per <= 8;
  const cudaError_t err = !window             ? launch_attn_tc(d, a, c, s)
                          : d.head_dim == 128 ? launch_d<128>(w, c, s)
                                              : launch_d<64>(w, c, s);
  trace_mark(MOE_KERNEL_ATTN, true, s);
  return err;
}

}  // namespace moe
