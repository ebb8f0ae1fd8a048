// Attention over the paged cache, small tiles of queries on the legacy tensor path (mma.sync).
//
// The query heads of a group share their key/value head, so that a tile's rows are (token, head of the group) pairs:
// row r is token r / G, head r % G.  One pass over the keys with the running maximum and sum of the softmax:
//   s_j = scale q.k_j,  m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),  o' = o e^(m - m') + ...
// in base 2 with scale * log2(e) folded in.  A CTA holds WM x WK warps: WM tiles of 16 rows, and each 64-key tile
// is shared out over WK warps, which keep their own m, l, o and join them at the end.  Keys and values come by
// cp.async in 64-key stages (rows of the page table looked up per copy, rows that no query of the tile sees filled
// with zeros, so that nothing behind them can reach an output).
#include <algorithm>

#include "attn.cuh"
#include "sync.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;         // keys a stage
constexpr int kLogBK = 6;
constexpr int kWinStages = 3;
constexpr int kWave = 296;      // CTAs aimed at when a window's keys are split: two a SM

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
// 16 bytes to shared memory, zeros when !ok.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

template <int D, int WM, int WK>
struct WinCfg {
  static constexpr int kThreads = WM * WK * 32;
  static constexpr int kRows = 16 * WM;
  static constexpr int kKeys = kBK / WK;            // keys a warp
  static constexpr int kTileBytes = kBK * D * 2;    // K or V of a stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kSmem = kWinStages * kStageBytes;
  static_assert(WK == 1 || WK * kRows * (D + 2) * 4 <= kSmem, "the warps' join reuses the stages");
};

struct WinArgs {
  AttnArgs a;
  int row_tiles, splits;
};

template <int D, int WM, int WK>
__global__ void __launch_bounds__(WinCfg<D, WM, WK>::kThreads) attn_mma_kernel(const __grid_constant__ WinArgs w) {
  using C = WinCfg<D, WM, WK>;
  constexpr int kChunks = D / 8;  // 16-byte pieces a row
  extern __shared__ __align__(128) uint8_t win_smem[];
  __shared__ uint32_t bad_v[kBK / 32];
  const AttnArgs &a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int wm = warp % WM, wk = warp / WM;
  int u = blockIdx.x;
  const int split = u % w.splits;
  u /= w.splits;
  const int rt = u % w.row_tiles;
  u /= w.row_tiles;
  const int hv = u % a.V, b = u / a.V;

  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
  const SeqView s = seq_view(a.kv.q_start, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
  const int rows = s.m * a.G, r0 = rt * C::kRows;
  if (r0 >= rows) return;
  const int base = s.n - s.m;  // position of new token 0
  const int p0 = base + r0 / a.G, p1 = base + (min(rows, r0 + C::kRows) - 1) / a.G;
  const TileRange tr = tile_range(p0, p1, s.n, a.window, a.n_sinks, kLogBK);
  const int t_lo = (int)((long long)tr.count * split / w.splits), t_hi = (int)((long long)tr.count * (split + 1) / w.splits);
  const int32_t *table = a.kv.table + (size_t)b * a.kv.max_pages;

  // the queries of this warp's 16 rows, as A fragments
  const int ra = r0 + 16 * wm + g, rb = ra + 8;
  const int pa = ra < rows ? base + ra / a.G : -1, pb = rb < rows ? base + rb / a.G : -1;
  const uint16_t *qa = a.q + (size_t)(s.q0 + ra / a.G) * a.ld_q + (size_t)(hv * a.G + ra % a.G) * D;
  const uint16_t *qb = a.q + (size_t)(s.q0 + rb / a.G) * a.ld_q + (size_t)(hv * a.G + rb % a.G) * D;
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    qf[k][0] = ra < rows ? __ldg(reinterpret_cast<const uint32_t *>(qa + 16 * k + 2 * c)) : 0u;
    qf[k][1] = rb < rows ? __ldg(reinterpret_cast<const uint32_t *>(qb + 16 * k + 2 * c)) : 0u;
    qf[k][2] = ra < rows ? __ldg(reinterpret_cast<const uint32_t *>(qa + 16 * k + 8 + 2 * c)) : 0u;
    qf[k][3] = rb < rows ? __ldg(reinterpret_cast<const uint32_t *>(qb + 16 * k + 8 + 2 * c)) : 0u;
  }

  const uint32_t smem0 = smem_u32(win_smem);
  auto load = [&](int t) {
    if (t < t_hi) {
      const int j0 = tile_of(tr, t) << kLogBK;
      const uint32_t st = smem0 + (uint32_t)((t - t_lo) % kWinStages) * C::kStageBytes;
      for (int i = threadIdx.x; i < kBK * kChunks; i += C::kThreads) {
        const int r = i / kChunks, ch = i % kChunks, j = j0 + r;
        // seen by the first or the last query that could: the visible set of a query grows at one end and
        // shrinks at the other, so that a key in neither is in none between them
        bool ok = j <= p1 && j < s.n && (a.window <= 0 || p0 - j < a.window || j < a.n_sinks);
        int64_t row = -1;
        if (ok) row = cache_row(table, j, a.kv.log_ps, a.kv.n_pages, a.V);
        ok = ok && row >= 0;
        const size_t off = ok ? ((size_t)row + ((size_t)hv << a.kv.log_ps)) * D + (size_t)ch * 8 : 0;
        const uint32_t dst = st + (uint32_t)(r * kChunks + (ch ^ (r & 7))) * 16u;
        cp_async16_or_zero(dst, a.k + off, ok);
        cp_async16_or_zero(dst + C::kTileBytes, a.v + off, ok);
      }
    }
    cp_async_commit();
  };

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

#pragma unroll
  for (int i = 0; i < kWinStages - 1; ++i) load(t_lo + i);
  for (int t = t_lo; t < t_hi; ++t) {
    cp_async_wait_group<kWinStages - 2>();
    __syncthreads();
    load(t + kWinStages - 1);
    const int j0 = tile_of(tr, t) << kLogBK;
    const uint32_t st = smem0 + (uint32_t)((t - t_lo) % kWinStages) * C::kStageBytes;
    // every key of the tile is seen by every row and lies in a valid page: no masks
    bool full = tile_full(p0, p1, j0, kBK, s.n, a.window, a.n_sinks);
    for (int p = j0 >> a.kv.log_ps; full && p <= (j0 + kBK - 1) >> a.kv.log_ps; ++p) {
      const int32_t page = __ldg(table + p);
      full = page >= 0 && page < a.kv.n_pages;
    }
    if (!full) {
      // A key that only some of the rows see: 0 * v is NaN when v is not finite, so such rows of V are cleared and
      // the rows that do see them become NaN.
      uint8_t *vt = win_smem + ((t - t_lo) % kWinStages) * C::kStageBytes + C::kTileBytes;
      if (threadIdx.x < kBK / 32) bad_v[threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < kBK * kChunks; i += C::kThreads) {
        const uint4 x = *reinterpret_cast<const uint4 *>(vt + (size_t)i * 16);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          bad |= (v[e] & 0x7f80u) == 0x7f80u || (v[e] & 0x7f800000u) == 0x7f800000u;
        if (bad) {
          const int r = i / kChunks;
          atomicOr(&bad_v[r >> 5], 1u << (r & 31));
        }
      }
      __syncthreads();
      if (bad_v[0] | bad_v[1]) {
        for (int i = threadIdx.x; i < kBK * kChunks; i += C::kThreads) {
          const int r = i / kChunks;
          if (bad_v[r >> 5] >> (r & 31) & 1) *reinterpret_cast<uint4 *>(vt + (size_t)i * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
      }
    }

    float sc[C::kKeys / 8][4];
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
    const int key0 = wk * C::kKeys;
#pragma unroll
    for (int n = 0; n < C::kKeys / 16; ++n) {
      const int r = key0 + 16 * n + (lane & 7) + ((lane & 16) ? 8 : 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int ch = 2 * k + ((lane >> 3) & 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(st + (uint32_t)(r * kChunks + (ch ^ (r & 7))) * 16u, b0, b1, b2, b3);
        mma_bf16_16816(sc[2 * n], qf[k], b0, b1, sc[2 * n]);
        mma_bf16_16816(sc[2 * n + 1], qf[k], b2, b3, sc[2 * n + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] *= a.scale_log2;
    bool nan_a = false, nan_b = false;
    if (!full) {
#pragma unroll
      for (int i = 0; i < C::kKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int jj = key0 + 8 * i + 2 * c + e, j = j0 + jj;
          const bool in = j < s.n && cache_row(table, j, a.kv.log_ps, a.kv.n_pages, a.V) >= 0;
          const bool va = in && key_seen(pa, j, s.n, a.window, a.n_sinks);
          const bool vb = in && key_seen(pb, j, s.n, a.window, a.n_sinks);
          const bool bad = bad_v[jj >> 5] >> (jj & 31) & 1;
          nan_a |= bad && va;
          nan_b |= bad && vb;
          if (j < s.n && !in && (va || vb || key_seen(pa, j, s.n, a.window, a.n_sinks) || key_seen(pb, j, s.n, a.window, a.n_sinks)))
            set_status(a.status, kStatusBadIndex);
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
    const float fa = exp2f(ma - sa), fb = exp2f(mb - sb);
    ma = na;
    mb = nb;
    float ta = nan_a ? NAN : 0.f, tb = nan_b ? NAN : 0.f;
    uint32_t pf[C::kKeys / 8][2];
#pragma unroll
    for (int i = 0; i < C::kKeys / 8; ++i) {
      const float e0 = exp2f(sc[i][0] - sa), e1 = exp2f(sc[i][1] - sa);
      const float e2 = exp2f(sc[i][2] - sb), e3 = exp2f(sc[i][3] - sb);
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
    for (int n = 0; n < C::kKeys / 16; ++n) {
      const uint32_t af[4] = {pf[2 * n][0], pf[2 * n][1], pf[2 * n + 1][0], pf[2 * n + 1][1]};
      const int r = key0 + 16 * n + (lane & 15);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const int ch = 2 * d + (lane >> 4);
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(st + C::kTileBytes + (uint32_t)(r * kChunks + (ch ^ (r & 7))) * 16u, b0, b1, b2, b3);
        mma_bf16_16816(o[2 * d], af, b0, b1, o[2 * d]);
        mma_bf16_16816(o[2 * d + 1], af, b2, b3, o[2 * d + 1]);
      }
    }
  }
  cp_async_wait_all();
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, d);
    lb += __shfl_xor_sync(0xffffffffu, lb, d);
  }

  // join the WK warps of each row tile: parts to shared memory, summed in warp order
  float *os = reinterpret_cast<float *>(win_smem);               // [WK][rows][D]
  float *ms = os + (size_t)WK * C::kRows * D;                    // [WK][rows] maximum, then sum
  __syncthreads();
  const int rl = wk * C::kRows + 16 * wm + g;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    *reinterpret_cast<float2 *>(os + (size_t)rl * D + 8 * i + 2 * c) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2 *>(os + (size_t)(rl + 8) * D + 8 * i + 2 * c) = make_float2(o[i][2], o[i][3]);
  }
  if (c == 0) {
    ms[2 * rl] = ma;
    ms[2 * rl + 1] = la;
    ms[2 * (rl + 8)] = mb;
    ms[2 * (rl + 8) + 1] = lb;
  }
  __syncthreads();
  float *po = a.part + (size_t)blockIdx.x * C::kRows * (D + 2), *pm = po + (size_t)C::kRows * D;
  for (int i = threadIdx.x; i < C::kRows * (D / 2); i += C::kThreads) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2)), rg = r0 + r;
    if (rg >= rows) continue;
    float m = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
    for (int k = 0; k < WK; ++k) m = fmaxf(m, ms[2 * (k * C::kRows + r)]);
    const float sub = m == -INFINITY ? 0.f : m;
    for (int k = 0; k < WK; ++k) {
      const float f = exp2f(ms[2 * (k * C::kRows + r)] - sub);
      const float2 v = *reinterpret_cast<const float2 *>(os + (size_t)(k * C::kRows + r) * D + d);
      l += f * ms[2 * (k * C::kRows + r) + 1];
      x += f * v.x;
      y += f * v.y;
    }
    if (w.splits == 1) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      uint16_t *dst = a.out + ((size_t)(s.q0 + rg / a.G) * a.H + (size_t)hv * a.G + rg % a.G) * D + d;
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(x * inv, y * inv);
    } else {
      *reinterpret_cast<float2 *>(po + (size_t)r * D + d) = make_float2(x, y);
      if (d == 0) {
        pm[2 * r] = m;
        pm[2 * r + 1] = l;
      }
    }
  }
}

// The parts of each row in split order: one CTA a (sequence, key/value head, row tile).
template <int D, int ROWS>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ WinArgs w) {
  const AttnArgs &a = w.a;
  int u = blockIdx.x;
  const int rt = u % w.row_tiles;
  u /= w.row_tiles;
  const int hv = u % a.V, b = u / a.V;
  const SeqView s = seq_view(a.kv.q_start, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
  const int rows = s.m * a.G, r0 = rt * ROWS;
  for (int i = threadIdx.x; i < ROWS * (D / 2); i += blockDim.x) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2)), rg = r0 + r;
    if (rg >= rows) continue;
    const float *p = a.part + (size_t)blockIdx.x * w.splits * ROWS * (D + 2);
    float m = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
    for (int k = 0; k < w.splits; ++k) m = fmaxf(m, p[(size_t)k * ROWS * (D + 2) + ROWS * D + 2 * r]);
    const float sub = m == -INFINITY ? 0.f : m;
    for (int k = 0; k < w.splits; ++k) {
      const float *pk = p + (size_t)k * ROWS * (D + 2);
      const float f = exp2f(pk[ROWS * D + 2 * r] - sub);
      const float2 v = *reinterpret_cast<const float2 *>(pk + (size_t)r * D + d);
      l += f * pk[ROWS * D + 2 * r + 1];
      x += f * v.x;
      y += f * v.y;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t *dst = a.out + ((size_t)(s.q0 + rg / a.G) * a.H + (size_t)hv * a.G + rg % a.G) * D + d;
    *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(x * inv, y * inv);
  }
}

template <int D, int WM, int WK>
cudaError_t launch(WinArgs w, bool window, cudaStream_t s) {
  using C = WinCfg<D, WM, WK>;
  const int per = w.a.kv.q_start ? w.a.T : w.a.kv.per;
  w.row_tiles = (int)(((long long)per * w.a.G + C::kRows - 1) / C::kRows);
  const long long units = (long long)w.a.kv.n_seqs * w.a.V * w.row_tiles;
  w.splits = window ? (int)std::max(1ll, kWave / units) : 1;
  if (units * w.splits > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(attn_mma_kernel<D, WM, WK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  attn_mma_kernel<D, WM, WK><<<(unsigned)(units * w.splits), C::kThreads, C::kSmem, s>>>(w);
  err = cudaGetLastError();
  if (err == cudaSuccess && w.splits > 1) {
    attn_join_kernel<D, C::kRows><<<(unsigned)units, 256, 0, s>>>(w);
    err = cudaGetLastError();
  }
  return err;
}

template <int D>
cudaError_t launch_d(const WinArgs &w, cudaStream_t s) {
  const bool window = !w.a.kv.q_start && w.a.kv.per <= 8;
  const int rows = w.a.kv.per * w.a.G;
  if (window && rows <= 16) return launch<D, 1, 4>(w, true, s);
  if (window && rows <= 32) return launch<D, 2, 2>(w, true, s);
  return launch<D, 4, 1>(w, window, s);
}

}  // namespace

// Parts exist only where a window is split, in at most kWave CTAs of at most 64 rows.
size_t attn_part_bytes(const moe_attn_dims &d, int, int) { return (size_t)kWave * 64 * (d.head_dim + 2) * 4; }

cudaError_t launch_attn(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s) {
  WinArgs w{a, 1, 1};
  trace_mark(MOE_KERNEL_ATTN, false, s);
  const bool window = !a.kv.q_start && a.kv.per <= 8;
  const cudaError_t err = !window             ? launch_attn_tc(d, a, c, s)
                          : d.head_dim == 128 ? launch_d<128>(w, s)
                                              : launch_d<64>(w, s);
  trace_mark(MOE_KERNEL_ATTN, true, s);
  return err;
}

}  // namespace moe
