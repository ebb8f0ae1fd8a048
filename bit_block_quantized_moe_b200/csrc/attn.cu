// Attention of verify windows (1 to 8 new tokens a sequence) over the paged cache, on the legacy tensor path
// (mma.sync): the work is reading the cache once, and a window's few rows fill 16-row products, not 128-row ones.
//
// The query heads of a group share their key/value head, so that a tile's rows are (token, head of the group) pairs:
// row r is token r / G, head r % G.  One pass over the keys with the running maximum and sum of the softmax:
//   s_j = scale q.k_j,  m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),  o' = o e^(m - m') + ...
// in base 2 with scale * log2(e) folded in.
//
// Split: all key tiles of all (sequence, key/value head, row tile) groups stand in one line, which is cut into
// equal shares whatever the lengths (they are read on the device, so that a captured graph follows them).  With work
// for more than one share a CTA, the CTAs take the later shares as they come free.  A group that is cut leaves parts
// (m, l, o) in the workspace; the CTA that brings the last one joins them in share order, so that the result does not
// depend on which that is.
//   last warp  : walks the line; TMA of K and V, a page at a time, into a ring of stages (128-byte swizzle); a group's
//                queries, and a record of where the stage stands, beside it;
//   8 warps    : the scores of 1/8 of the keys each, the weights to shared memory, then D/8 columns of the output each
//                over all keys.  A warp's output is few registers, which leaves room for two CTAs a SM (one waits
//                while the other computes), and a group's end needs no exchange but of the row sums.  The running
//                maximum is left as it is until some score exceeds it by 8 (a factor of 256, which fp32 sums and bf16
//                weights carry without loss), so that a tile needs one meeting of the warps, which also tells them
//                whether it is so.
// Rows of V that no query of the window sees are masked in the registers that feed the product, so that nothing behind
// them can reach an output.  Every wait is bounded (sync.cuh).
#include <algorithm>

#include "attn.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kMinTiles = 1;     // tiles that a share has at least
constexpr int kShareTiles = 16;  // tiles that a share has at least where there are several a CTA
constexpr float kWinLazy = 8.0f;

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
// Arrives on `bar` once this thread's earlier cp.async copies have landed (one of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, int MT>
struct WinCfg {
  static constexpr int kLogBK = D == 128 ? 6 : 7;   // keys a tile: 16 KB of K and of V
  static constexpr int kBK = 1 << kLogBK;
  static constexpr int kWarps = 8;                  // beside the producer
  static constexpr int kNK = kBK / 64;              // 8-key groups a warp
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kRows = 16 * MT;
  static constexpr int kCtas = MT == 1 ? 2 : 1;     // a SM
  static constexpr int kHalfBytes = kBK * 128;      // 64 columns of a tile, one swizzle row a key
  static constexpr int kTileBytes = kBK * D * 2;    // K or V of a stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = MT == 1 ? 3 : MT == 2 ? 5 : 4;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQAt = kStages * kStageBytes;
  static constexpr int kPAt = kQAt + kStages * kQBytes;
  static constexpr int kPBytes = kRows * kBK * 2;
  static constexpr int kSmem = kPAt + 2 * kPBytes;  // weights by turns: a warp may be one tile ahead
};

constexpr int kRecFirst = 1, kRecLast = 2;  // of this CTA's part of the group
constexpr int kRecPartial = 4;               // some row does not see some key of the tile
constexpr int kRecEnd = 8;                   // no tile: the CTA is done

// What the producer tells beside a stage.
struct TileRec {
  int b, hv, rt;      // the group: sequence, key/value head, row tile
  int j0, n;          // first key of the tile, keys of the sequence
  int q;              // with `first`: which of the places holds the group's queries
  int flags;          // kRec...
  int share, c0, c1;  // this share, and the shares that hold the group
  int slot, slot0;    // where this share's part lies, and where that of c0 does
  uint32_t bad[4];    // keys whose page is outside the cache
};

template <int STAGES>
struct WinBars {
  uint64_t full[STAGES], empty[STAGES];
  TileRec rec[STAGES];
  int abort;
};

struct WinArgs {
  AttnArgs a;
  int row_tiles;
};

// The key tiles of a sequence; one in which nothing is seen where it is empty.
__device__ __forceinline__ TileRange window_tiles(const AttnArgs &a, const SeqView &s, int log_bk) {
  TileRange r = tile_range(s.n - s.m, s.n - 1, s.n, a.window, a.n_sinks, log_bk);
  if (r.count < 1) r.count = 1;
  return r;
}

__device__ __forceinline__ int window_count(const AttnArgs &a, int b, int log_bk) {
  if (b >= a.kv.n_seqs) return 0;
  return window_tiles(a, seq_view(nullptr, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap), log_bk).count;
}

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

// floor(a * b / c) for a >= 0, small b and c > 0; in 32 bits where they hold it, which is many times quicker.
__device__ __forceinline__ long long mul_div(long long a, int b, int c) {
  const unsigned long long p = (unsigned long long)a * b;
  return p >> 32 ? (long long)(p / c) : (long long)((uint32_t)p / (uint32_t)c);
}

// The share that holds tile x: the largest i with total * i / shares <= x.
__device__ __forceinline__ int share_of(long long x, int shares, long long total) {
  const unsigned long long p = (unsigned long long)(x + 1) * shares - 1;
  return p >> 32 ? (int)(p / total) : (int)((uint32_t)p / (uint32_t)total);
}

// Shares of a line of `total` tiles in `count` groups on `ctas` CTAs.
__device__ __forceinline__ int share_count(long long total, long long count, int ctas) {
  const long long least = (total + kMinTiles - 1) / kMinTiles;
  if (least <= ctas) return (int)least;
  if (count * 2 < ctas) return ctas;
  return ctas * (int)min((long long)(kAttnShares / ctas), max(1ll, total / ((long long)ctas * kShareTiles)));
}

// Whether 16 bytes hold a bf16 infinity or NaN.
__device__ __forceinline__ bool not_finite8(const uint4 &x) {
  const uint32_t e[4] = {x.x, x.y, x.z, x.w};
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) bad |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

// The computing warps meet; whether any thread came with `flag`.
__device__ __forceinline__ bool win_meet(bool flag, int threads) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)flag), "r"(threads)
      : "memory");
  return any != 0;
}

template <int D, int MT>
__global__ void __launch_bounds__(WinCfg<D, MT>::kThreads, WinCfg<D, MT>::kCtas)
    attn_window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ WinArgs w) {
  using C = WinCfg<D, MT>;
  constexpr int kChunks = D / 8;   // 16-byte pieces a row
  constexpr int kNT = D / 64;      // 8-column tiles of a warp's output
  extern __shared__ __align__(1024) uint8_t win_smem[];
  __shared__ WinBars<C::kStages> B;
  __shared__ long long sum_s[C::kThreads / 32];
  __shared__ __align__(16) float row_s[C::kRows][C::kWarps];  // maxima, or sums, of each row by warp
  __shared__ __align__(16) uint8_t use_s[2][16];  // by turns: a warp may be one tile ahead
  __shared__ int last_s;
  const AttnArgs &a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int groups = a.V * w.row_tiles, rows = a.kv.per * a.G;
  const uint32_t smem0 = smem_u32(win_smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 33);  // the producer's expected bytes, and its lanes' copies of queries
      mbar_init(&B.empty[i], C::kWarps);
    }
    B.abort = 0;
    mbar_fence_init();
  }

  // ---- the length of the line, and its shares
  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
  long long total = 0;
  for (int b = threadIdx.x; b < a.kv.n_seqs; b += C::kThreads) total += window_count(a, b, C::kLogBK);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sum_s[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < C::kThreads / 32; ++i) total += sum_s[i];
  total *= groups;
  const int shares = share_count(total, (long long)a.kv.n_seqs * groups, gridDim.x);
  if ((int)blockIdx.x >= shares) return;

  if (warp == C::kWarps) {
    // ---- producer: all but the pieces is uniform over the warp ----
    // lane l < pieces has piece l of a tile: a page, or half of one of 128
    const int log_pc = min(a.kv.log_ps, C::kLogBK), pc = 1 << log_pc, pieces = C::kBK >> log_pc;
    int st = 0, qn = 0, b = 0, share = blockIdx.x;
    uint32_t ph = 1;
    long long issued = 0, line = 0;  // line: tiles before sequence b
    bool live = true;
    while (live && share < shares) {
      // the next share, if there are more than CTAs: taken now, needed at this one's end
      uint32_t claim = 0;
      if (shares > (int)gridDim.x && lane == 0) claim = atomicAdd(a.counts + kAttnShares, 1u);
      const long long x0 = mul_div(total, share, shares), x1 = mul_div(total, share + 1, shares);
      // the sequence of x0: at or after the last share's
      for (;;) {
        long long incl = window_count(a, b + lane, C::kLogBK);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t beyond = __ballot_sync(0xffffffffu, line + incl * groups > x0);
        const int at = beyond ? __ffs(beyond) - 1 : 32;
        const long long skipped = __shfl_sync(0xffffffffu, incl, at > 0 ? at - 1 : 0);
        if (at > 0) line += skipped * groups;
        b += at;
        if (beyond || b >= a.kv.n_seqs) break;
      }
      if (b >= a.kv.n_seqs) break;  // only where the lengths change under the call
      SeqView s = seq_view(nullptr, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
      TileRange r = window_tiles(a, s, C::kLogBK);
      const int gi = (int)mul_div(x0 - line, 1, r.count);
      int t = (int)(x0 - line - (long long)gi * r.count);
      int hv = gi / w.row_tiles, rt = gi - hv * w.row_tiles;
      // this lane's piece of the tile at the cursor
      auto piece = [&](bool &seen) {
        const int a0 = (tile_of(r, t) << C::kLogBK) + (lane << log_pc), e0 = a0 + pc;
        seen = lane < pieces && a0 < s.n && (a.window <= 0 || e0 - 1 > s.n - s.m - a.window || a0 < a.n_sinks);
        return seen ? __ldg(a.kv.table + (size_t)b * a.kv.max_pages + (a0 >> a.kv.log_ps)) : 0;
      };
      bool seen;
      int page = piece(seen);
      for (long long x = x0; x < x1; ++x) {
        live = __all_sync(0xffffffffu, win_wait(&B.empty[st], ph, B, a.status));
        if (!live) break;
        const bool ok = seen && page >= 0 && page < a.kv.n_pages;
        const uint32_t good = __ballot_sync(0xffffffffu, ok), wrong = __ballot_sync(0xffffffffu, seen && !ok);
        const bool first = x == x0 || t == 0;
        const int j0 = tile_of(r, t) << C::kLogBK, cb = b, chv = hv, crt = rt;
        // below 2^31: checked on the host
        const int row = ((page * a.V + hv) << a.kv.log_ps) + ((j0 + (lane << log_pc)) & ((1 << a.kv.log_ps) - 1));
        if (lane == 0) {
          TileRec &rec = B.rec[st];
          const bool last = x + 1 == x1 || t + 1 == r.count;
          rec.b = b;
          rec.hv = hv;
          rec.rt = rt;
          rec.j0 = j0;
          rec.n = s.n;
          rec.q = qn;
          rec.flags = (first ? kRecFirst : 0) | (last ? kRecLast : 0) |
                      (wrong || !tile_full(s.n - s.m, s.n - 1, j0, C::kBK, s.n, a.window, a.n_sinks) ? kRecPartial : 0);
          if (last) {
            const long long gs = x - t, ge = gs + r.count;
            rec.share = share;
            rec.c0 = gs >= x0 ? share : share_of(gs, shares, total);
            rec.c1 = ge <= x1 ? share : share_of(ge - 1, shares, total);
            rec.slot = gs > x0;
            rec.slot0 = gs > (gs >= x0 ? x0 : mul_div(total, rec.c0, shares));
          }
          rec.bad[0] = rec.bad[1] = rec.bad[2] = rec.bad[3] = 0;
          if (wrong) {
            for (int k = 0; k < C::kBK; ++k)
              if (wrong >> (k >> log_pc) & 1) rec.bad[k >> 5] |= 1u << (k & 31);
            set_status(a.status, kStatusBadIndex);
          }
          mbar_arrive_expect_tx(&B.full[st], (uint32_t)(__popc(good) * pc * D * 4));
        }
        __syncwarp();
        if (ok) {
          uint8_t *dst = win_smem + st * C::kStageBytes + lane * pc * 128;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            tma_load_2d(dst + h * C::kHalfBytes, &kmap, h * 64, row, &B.full[st]);
            tma_load_2d(dst + C::kTileBytes + h * C::kHalfBytes, &vmap, h * 64, row, &B.full[st]);
          }
        }
        __syncwarp();
        // the cursor, and the next tile's pages, which come in while this warp waits for a stage
        if (++t == r.count) {
          t = 0;
          if (++rt == w.row_tiles) {
            rt = 0;
            if (++hv == a.V) {
              hv = 0;
              if (x + 1 < x1) {
                line += (long long)r.count * groups;
                s = seq_view(nullptr, a.kv.kv_len, ++b, a.kv.per, a.T, a.kv.cap);
                r = window_tiles(a, s, C::kLogBK);
              }
            }
          }
        }
        if (x + 1 < x1) page = piece(seen);
        if (first) {
          // the group's queries; rows behind the last are zeros.  The groups in flight are no more than the stages,
          // so that as many places in turn suffice.
          const uint32_t dst = smem0 + C::kQAt + (uint32_t)qn * C::kQBytes;
          qn = qn + 1 == C::kStages ? 0 : qn + 1;
          for (int i = lane; i < C::kRows * kChunks; i += 32) {
            const int rr = i / kChunks, ch = i % kChunks, rg = crt * C::kRows + rr, tok = rg / a.G;
            const bool in = rg < rows;
            const uint16_t *src = a.q + (in ? (size_t)(cb * a.kv.per + tok) * a.ld_q + (size_t)(chv * a.G + rg - tok * a.G) * D + ch * 8 : 0);
            cp_async16_or_zero(dst + (uint32_t)(rr * kChunks + (ch ^ (rr & 7))) * 16u, src, in);
          }
        }
        cp_async_arrive(&B.full[st]);  // every lane, when its copies have landed
        ++issued;
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
      if (shares <= (int)gridDim.x) break;
      claim = __shfl_sync(0xffffffffu, claim, 0);
      share = gridDim.x + claim;
      // every CTA makes one claim that finds nothing; the very last claim leaves the counter ready for the next call
      if (lane == 0 && claim == (uint32_t)(shares - 1)) a.counts[kAttnShares] = 0;
    }
    // The end record takes the oldest stage, whose tile has been read.
    const bool told = __all_sync(0xffffffffu, win_wait(&B.empty[st], ph, B, a.status));
    if (told) {
      if (lane == 0) {
        B.rec[st].flags = kRecEnd;
        mbar_arrive(&B.full[st]);
      }
      __syncwarp();
      mbar_arrive(&B.full[st]);
    }
    // every copy issued must land before the CTA exits, also after an abort
    const int open = C::kStages - (told ? 1 : 0);
    for (long long i = issued > open ? issued - open : 0; i < issued; ++i)
      if (!mbar_wait(&B.full[i % C::kStages], (uint32_t)(i / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
    return;
  }

  // ---- the other warps ----
  constexpr int kMeet = C::kWarps * 32;
  uint32_t phase = 0;
  int cs = 0, turn = 0;
  uint32_t qf[MT == 1 ? D / 16 : 1][4];  // a single row tile's queries stay in registers
  float o[MT][kNT][4], m[MT][2], l[MT][2];
  uint32_t qs = 0;                       // where the group's queries lie
  for (;;) {
    const bool came = win_wait(&B.full[cs], phase, B, a.status);
    const TileRec &rec = B.rec[cs];
    const int flags = came ? rec.flags : kRecEnd;
    const uint32_t st = smem0 + (uint32_t)cs * C::kStageBytes, ps = smem0 + C::kPAt + (uint32_t)turn * C::kPBytes;
    float sc[MT][C::kNK][4];
    bool grow = flags & kRecEnd;
    if (!grow) {
      if (flags & kRecFirst) {
        qs = smem0 + C::kQAt + (uint32_t)rec.q * C::kQBytes;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int t = 0; t < kNT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
          m[i][0] = m[i][1] = -INFINITY;
          l[i][0] = l[i][1] = 0.f;
        }
        if constexpr (MT == 1) {
          const int r = lane & 15;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            ldsm_x4(qs + (uint32_t)(r * kChunks + ((2 * k + (lane >> 4)) ^ (r & 7))) * 16u, qf[k][0], qf[k][1], qf[k][2],
                    qf[k][3]);
        }
      }
      // ---- scores of this warp's keys
#pragma unroll
      for (int nk = 0; nk < C::kNK; ++nk) {
        uint32_t kf[D / 16][2];
        const int r = 8 * (C::kNK * warp + nk) + (lane & 7);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const int ch = 4 * k + (lane >> 3);
          ldsm_x4(st + (uint32_t)((ch >> 3) * C::kHalfBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4)), kf[2 * k][0],
                  kf[2 * k][1], kf[2 * k + 1][0], kf[2 * k + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t af[4];
            if constexpr (MT == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) af[e] = qf[k][e];
            } else {
              const int rq = 16 * i + (lane & 15);
              ldsm_x4(qs + (uint32_t)(rq * kChunks + ((2 * k + (lane >> 4)) ^ (rq & 7))) * 16u, af[0], af[1], af[2], af[3]);
            }
            if (k & 1)
              mma_bf16_16816(s1, af, kf[k][0], kf[k][1], s1);
            else
              mma_bf16_16816(s0, af, kf[k][0], kf[k][1], s0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][nk][e] = (s0[e] + s1[e]) * a.scale_log2;
        }
      }
      if (flags & kRecPartial) {
        // which of the warp's keys some row sees, and of these the ones whose values are not finite: 0 * v is NaN
        // then, so that where rows differ in what they see such a key is left out of the product, and the rows that
        // see it become NaN
        const int n = rec.n, j0 = rec.j0, base_pos = n - a.kv.per, r0 = rec.rt * C::kRows;
#pragma unroll
        for (int nk = 0; nk < C::kNK; ++nk) {
          const int k0 = 8 * (C::kNK * warp + nk), kk = k0 + (lane >> 2), j = j0 + kk;
          const bool live = j < n && (a.window <= 0 || base_pos - j < a.window || j < a.n_sinks) &&
                            !(rec.bad[kk >> 5] >> (kk & 31) & 1);
          bool bad = false;
          if (live && a.kv.per > 1) {
            const uint8_t *v = win_smem + cs * C::kStageBytes + C::kTileBytes + kk * 128;
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i) {
              const int ch = 4 * i + (lane & 3);
              bad |= not_finite8(*reinterpret_cast<const uint4 *>(v + (ch >> 3) * C::kHalfBytes + (((ch & 7) ^ (kk & 7)) << 4)));
            }
          }
          const uint32_t lv = __ballot_sync(0xffffffffu, live);
          uint32_t bd = __ballot_sync(0xffffffffu, bad);  // a key's bits: lanes 4k .. 4k + 3
          bd |= bd >> 1;
          bd |= bd >> 2;
          uint32_t use = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) use |= ((lv & ~bd) >> (4 * k) & 1) << k;
          if (lane == 0) use_s[turn][C::kNK * warp + nk] = (uint8_t)use;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int rg = r0 + 16 * i + g + 8 * h;
              const int pos = rg < rows ? base_pos + rg / a.G : -1;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = 2 * c + e;
                const bool v = (lv >> (4 * key) & 1) && key_seen(pos, j0 + k0 + key, n, a.window, a.n_sinks);
                if (v && (bd >> (4 * key) & 1)) l[i][h] = NAN;
                if (!v) sc[i][nk][2 * h + e] = -INFINITY;
              }
            }
        }
      }
    }
    // ---- weights, with the maximum as it stands
    auto weights = [&](int i, int h) {
      const int r = 16 * i + g + 8 * h;
      const float sub = m[i][h] == -INFINITY ? 0.f : m[i][h];  // nothing seen yet: 2^(-inf - 0) = 0
      float sum = 0.f;
#pragma unroll
      for (int nk = 0; nk < C::kNK; ++nk) {
        const float e0 = ex2(sc[i][nk][2 * h] - sub), e1 = ex2(sc[i][nk][2 * h + 1] - sub);
        sum += e0 + e1;
        const int ch = C::kNK * warp + nk;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(ps + (uint32_t)(r * (2 * C::kBK) + ((ch ^ (r & 7)) << 4) + 4 * c)),
                     "r"(pack_bf16x2(e0, e1))
                     : "memory");
      }
      return sum;
    };
    float sums[MT][2];
    if (!(flags & kRecEnd)) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float most = m[i][h] + kWinLazy;
#pragma unroll
          for (int nk = 0; nk < C::kNK; ++nk) grow |= !(sc[i][nk][2 * h] <= most) || !(sc[i][nk][2 * h + 1] <= most);
          sums[i][h] = weights(i, h);
        }
    }
    // the meeting: the weights are there, unless a maximum has to grow (or the end has come)
    if (win_meet(grow, kMeet)) {
      if (win_meet(!came, kMeet) || (flags & kRecEnd)) break;  // all leave together when a wait has given up
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = fmaxf(sc[i][0][2 * h], sc[i][0][2 * h + 1]);
          if constexpr (C::kNK == 2) x = fmaxf(x, fmaxf(sc[i][C::kNK - 1][2 * h], sc[i][C::kNK - 1][2 * h + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          if (c == 0) row_s[16 * i + g + 8 * h][warp] = x;
        }
      win_meet(false, kMeet);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * i + g + 8 * h;
          const float4 x0 = *reinterpret_cast<const float4 *>(&row_s[r][0]), x1 = *reinterpret_cast<const float4 *>(&row_s[r][4]);
          const float mx = fmaxf(fmaxf(fmaxf(x0.x, x0.y), fmaxf(x0.z, x0.w)), fmaxf(fmaxf(x1.x, x1.y), fmaxf(x1.z, x1.w)));
          const float nm = fmaxf(m[i][h], mx);
          const float f = ex2(m[i][h] - (nm == -INFINITY ? 0.f : nm));
          m[i][h] = nm;
          l[i][h] *= f;
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            o[i][t][2 * h] *= f;
            o[i][t][2 * h + 1] *= f;
          }
          sums[i][h] = weights(i, h);
        }
      win_meet(false, kMeet);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      l[i][0] += sums[i][0];
      l[i][1] += sums[i][1];
    }
    // ---- products: V fragments of this warp's columns, two 16-key steps a round
#pragma unroll
    for (int k = 0; k < C::kBK / 16; k += 2) {
      uint32_t vf[2][kNT][2];
      if constexpr (kNT == 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * (k + e) + (lane & 15), ch = 2 * warp + (lane >> 4);
          ldsm_x4_t(st + (uint32_t)(C::kTileBytes + (ch >> 3) * C::kHalfBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                    vf[e][0][0], vf[e][0][1], vf[e][kNT - 1][0], vf[e][kNT - 1][1]);
        }
      } else {
        const int r = 16 * k + lane;
        ldsm_x4_t(st + (uint32_t)(C::kTileBytes + r * 128 + ((warp ^ (r & 7)) << 4)), vf[0][0][0], vf[0][0][1],
                  vf[1][0][0], vf[1][0][1]);
      }
      if (flags & kRecPartial) {
        const uint32_t use = *reinterpret_cast<const volatile uint32_t *>(&use_s[turn][2 * k]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // this lane's keys of the two halves of a fragment: 2c, 2c + 1 and 8 more
          const uint32_t u = use >> (16 * e + 2 * c);
          const uint32_t v0 = (u & 1 ? 0xffffu : 0u) | (u & 2 ? 0xffff0000u : 0u);
          const uint32_t v1 = (u & 256 ? 0xffffu : 0u) | (u & 512 ? 0xffff0000u : 0u);
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            vf[e][t][0] &= v0;
            vf[e][t][1] &= v1;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * i + (lane & 15);
          uint32_t af[4];
          ldsm_x4(ps + (uint32_t)(r * (2 * C::kBK) + (((2 * (k + e) + (lane >> 4)) ^ (r & 7)) << 4)), af[0], af[1], af[2], af[3]);
#pragma unroll
          for (int t = 0; t < kNT; ++t) mma_bf16_16816(o[i][t], af, vf[e][t][0], vf[e][t][1], o[i][t]);
        }
    }
    turn ^= 1;
    int share = 0, c0 = 0, c1 = 0, slot = 0, slot0 = 0, hv = 0, q0 = 0, r0 = 0;
    if (flags & kRecLast) {
      share = rec.share;
      c0 = rec.c0;
      c1 = rec.c1;
      slot = rec.slot;
      slot0 = rec.slot0;
      hv = rec.hv;
      q0 = rec.b * a.kv.per;
      r0 = rec.rt * C::kRows;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.empty[cs]);
    if (++cs == C::kStages) {
      cs = 0;
      phase ^= 1;
    }
    if (!(flags & kRecLast)) continue;

    // ---- the end of this CTA's part of the group: row sums over the warps, in warp order
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[i][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c == 0) row_s[16 * i + g + 8 * h][warp] = x;
      }
    win_meet(false, kMeet);
    const int live = min(rows - r0, C::kRows);
    constexpr size_t kPart = (size_t)C::kRows * (D + 2);
    float *po = a.part + ((size_t)share * 2 + slot) * kPart, *pm = po + (size_t)C::kRows * D;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * i + g + 8 * h, rg = r0 + r, col = warp * (8 * kNT) + 2 * c;
        if (r >= live) continue;
        const float4 x0 = *reinterpret_cast<const float4 *>(&row_s[r][0]), x1 = *reinterpret_cast<const float4 *>(&row_s[r][4]);
        const float sum = ((x0.x + x0.y) + (x0.z + x0.w)) + ((x1.x + x1.y) + (x1.z + x1.w));
        if (c0 == c1) {
          const float inv = sum == 0.f ? 0.f : 1.0f / sum;
          const int tok = rg / a.G;
          uint16_t *dst = a.out + ((size_t)(q0 + tok) * a.H + (size_t)hv * a.G + rg - tok * a.G) * D + col;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
            *reinterpret_cast<uint32_t *>(dst + 8 * t) = pack_bf16x2(o[i][t][2 * h] * inv, o[i][t][2 * h + 1] * inv);
        } else {
#pragma unroll
          for (int t = 0; t < kNT; ++t)
            __stcg(reinterpret_cast<float2 *>(po + (size_t)r * D + col + 8 * t), make_float2(o[i][t][2 * h], o[i][t][2 * h + 1]));
          if (warp == 0 && c == 0) __stcg(reinterpret_cast<float2 *>(pm + 2 * r), make_float2(m[i][h], sum));
        }
      }
    if (c0 == c1) continue;
    // each share is the first of at most one cut group, whose count it keeps
    win_meet(false, kMeet);
    if (threadIdx.x == 0) {
      // releases the whole CTA's part (ordered before it by the meeting), acquires the others'
      uint32_t before;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.counts + c0) : "memory");
      last_s = before == (uint32_t)(c1 - c0);
      if (last_s) a.counts[c0] = 0;  // for the next call
    }
    win_meet(false, kMeet);
    if (!last_s) continue;
    for (int i = threadIdx.x; i < live * (D / 2); i += kMeet) {
      const int r = i / (D / 2), d = 2 * (i % (D / 2));
      float mm = -INFINITY, ll = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll 1
      for (int e0 = c0; e0 <= c1; e0 += 8) {
        float2 ml[8], v[8];  // eight parts in flight; behind the last one, the last with no weight
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = min(e0 + e, c1);
          const float *pk = a.part + ((size_t)k * 2 + (k == c0 ? slot0 : 0)) * kPart;
          ml[e] = __ldcg(reinterpret_cast<const float2 *>(pk + (size_t)C::kRows * D + 2 * r));
          v[e] = __ldcg(reinterpret_cast<const float2 *>(pk + (size_t)r * D + d));
        }
        float nm = mm;
#pragma unroll
        for (int e = 0; e < 8; ++e) nm = fmaxf(nm, ml[e].x);
        const float u = nm == -INFINITY ? 0.f : nm, f0 = ex2(mm - u);
        mm = nm;
        ll *= f0;
        y0 *= f0;
        y1 *= f0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e0 + e > c1) continue;
          const float f = ex2(ml[e].x - u);
          ll += ml[e].y * f;
          y0 += v[e].x * f;
          y1 += v[e].y * f;
        }
      }
      const float inv = ll == 0.f ? 0.f : 1.0f / ll;
      const int rg = r0 + r, tok = rg / a.G;
      uint16_t *dst = a.out + ((size_t)(q0 + tok) * a.H + (size_t)hv * a.G + rg - tok * a.G) * D + d;
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(y0 * inv, y1 * inv);
    }
  }
}

template <int D, int MT>
cudaError_t launch(WinArgs w, const moe_kv_cache &c, cudaStream_t s) {
  using C = WinCfg<D, MT>;
  CUtensorMap km, vm;
  if (!make_pages_map(&km, c.k, c.n_pages, w.a, D, C::kBK) ||
      !make_pages_map(&vm, c.v, c.n_pages, w.a, D, C::kBK))
    return cudaErrorInvalidValue;
  w.row_tiles = (w.a.kv.per * w.a.G + C::kRows - 1) / C::kRows;
  cudaError_t err = cudaFuncSetAttribute(attn_window_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  attn_window_kernel<D, MT><<<kAttnSms * C::kCtas, C::kThreads, C::kSmem, s>>>(km, vm, w);
  return cudaGetLastError();
}

// Rows of a window: one, two or four 16-row tiles side by side; more rows than 64 walk the keys again.
template <int D>
cudaError_t launch_d(const WinArgs &w, const moe_kv_cache &c, cudaStream_t s) {
  const int rows = w.a.kv.per * w.a.G;
  return rows <= 16 ? launch<D, 1>(w, c, s) : rows <= 32 ? launch<D, 2>(w, c, s) : launch<D, 4>(w, c, s);
}

}  // namespace

bool make_pages_map(CUtensorMap *map, const uint16_t *cache, int n_pages, const AttnArgs &a, int D, int tile) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)n_pages * a.V << a.kv.log_ps};  // rows below 2^31
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)std::min(1 << a.kv.log_ps, tile)};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(cache), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t attn_part_bytes(const moe_attn_dims &d, int, int) {
  const int rows = 8 * d.n_heads / d.n_kv_heads;  // the most rows of a window, then those of a CTA
  return (size_t)kAttnShares * 2 * (rows <= 16 ? 16 : rows <= 32 ? 32 : 64) * (d.head_dim + 2) * 4;
}

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
