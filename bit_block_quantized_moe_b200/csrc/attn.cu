// Attention of verify windows (1 to 8 new tokens a sequence) over the paged cache, on the legacy tensor path
// (mma.sync): the work is reading the cache once, and a window's few rows fill products 8 rows wide, not 128.
//
// The query heads of a group share their key/value head, so that a tile's rows are (token, head of the group) pairs:
// row r is token r / G, head r % G.  One pass over the keys with the running maximum and sum of the softmax:
//   s_j = scale q.k_j,  m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),  o' = o e^(m - m') + ...
// in base 2 with scale * log2(e) folded in.  Both products have the keys or the head dimension on the 16-row side and
// the query rows on the 8-column side (S^T = K Q^T, O^T = V^T P^T).
//
// Split: all key tiles of all (sequence, key/value head) groups stand in one line, which is cut into equal
// shares, one a CTA, whatever the lengths (they are read on the device, so that a captured graph follows them).
// (Smaller shares taken as CTAs come free were slower: every share's ends cost more than the balance gave.)  A group
// that is cut leaves parts (m, l, o) in the workspace; the CTA that brings the last one joins them in share order, so
// that the result does not depend on which that is.  Few groups over long caches have many parts each, too many for one
// CTA to read: they are joined by a second launch, a CTA a row (one token at position 131072 of 2 key/value heads, 148
// parts a head: 47.5 us with the join in one CTA).
//   last warp  : walks the line; TMA of K and V, a page at a time, into a ring of stages (128-byte swizzle); a group's
//                queries, and a record of where the stage stands, beside it;
//   4 warps    : the scores of a quarter of the keys each, the weights to shared memory, then a quarter of the output's
//                columns each over all keys, so that a group's end needs no exchange but of the row sums (8 warps for
//                more than 16 rows, in two groups with half of the rows each; one group of four with all of them took
//                86 us for 32 x 3 tokens at 8192, this 72.5).  The running
//                maximum is left as it is until some score exceeds it by 8 (a factor of 256, which fp32 sums and bf16
//                weights carry without loss), so that a tile needs one meeting of the warps, which also tells them
//                whether it is so.  Two CTAs a SM (of 4 warps): one computes while the other waits.
// Bound: HBM; 64 ragged sequences of up to 16384 tokens (0.55 GB of keys and values) take 92 us, 93% of the copy rate.
// Short calls are chains of waits: 500 tokens of one sequence 8 us.
// Values of keys that no query of the window sees are masked in the registers that feed the product, so that nothing
// behind them can reach an output.  Every wait on memory is bounded (sync.cuh).
#include <algorithm>

#include "attn.cuh"
#include "half.cuh"

namespace moe {
namespace {

constexpr float kWinLazy = 8.0f;
constexpr int kJoinParts = 12;  // more parts a group go to the second launch (4: 7 sequences 36 us instead of 25)
// Windows of more than 32 rows go to the chunk kernel's tiles (32 x 8 tokens of 8 heads a group at 8192: 66 us there,
// 131 here when this kernel still walked the keys once for 32 rows each), and those of 17 to 32 where it has five parts
// or more for each group, a sequence and key/value head.  Measured with windows of 3 tokens and 8 heads of 128 a group,
// us there / here: 8 groups of 1000 tokens 12 / 17, of 4000 14 / 20, of 16000 23 / 30, ragged up to 4000 15 / 19, up to
// 16000 22 / 24; 24 groups of 4000 21 / 25, of 16000 48 / 57, ragged up to 4000 21 / 24, but up to 16000 46 / 42; 29
// groups 23 / 28, 57 / 66, 22 / 24, but 53 / 42.  More groups stay, as few or no parts cannot even out their lengths: 64
// ragged up to 16000 115 / 69, 128 217 / 135, though with equal ones they would be quicker there too (128 of 1000 20 /
// 29, of 4000 62 / 71, of 16000 219 / 235): the lengths are on the device.  16 rows or fewer stay as well (8 x 2 ragged
// up to 16384: 32 there, 21 here).
constexpr int kWinRows = 32, kWinFew = kAttnSms / 5;

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

template <int D, int NR>
struct WinCfg {
  static constexpr int kLogBK = D == 128 ? 6 : 7;   // keys a tile: 16 KB of K and of V
  static constexpr int kBK = 1 << kLogBK;
  static constexpr int kRG = NR <= 2 ? 1 : NR / 2;  // groups of four warps, each with its own rows
  static constexpr int kNR = NR / kRG;              // 8-row tiles a warp
  static constexpr int kWarps = 4 * kRG;            // beside the producer
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kMK = kBK / 64;              // 16-key tiles a warp
  static constexpr int kMD = D / 64;                // 16-column tiles of the output a warp
  static constexpr int kRows = 8 * NR;
  static constexpr int kCtas = NR <= 2 ? 2 : 1;     // a SM
  static constexpr int kStages = NR <= 2 ? 3 : 4;   // what the shared memory holds
  static constexpr int kHalfBytes = kBK * 128;      // 64 columns of a tile, one swizzle row a key
  static constexpr int kTileBytes = kBK * D * 2;    // K or V of a stage
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQAt = kStages * kStageBytes;
  static constexpr int kPAt = kQAt + kStages * kQBytes;
  static constexpr int kPBytes = NR * kBK * 16;     // weights [8-row tile][key][8 rows], bf16
  static constexpr int kSmem = kPAt + 2 * kPBytes;  // by turns: a warp may be one tile ahead
};

constexpr int kRecFirst = 1, kRecLast = 2;  // of this CTA's part of the group
constexpr int kRecPartial = 4;               // some row does not see some key of the tile
constexpr int kRecEnd = 8;                   // no tile: the CTA is done

// What the producer tells beside a stage.
struct TileRec {
  int b, hv;          // the group: sequence, key/value head
  int j0, n;          // first key of the tile, keys of the sequence
  int q;              // with `first`: which of the places holds the group's queries
  int flags;          // kRec...
  int c0, c1;         // the shares that hold the group
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
  int join_after;  // parts are joined by attn_join_kernel
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

template <int D, int NR>
__global__ void __launch_bounds__(WinCfg<D, NR>::kThreads, WinCfg<D, NR>::kCtas)
    attn_window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ WinArgs w) {
  using C = WinCfg<D, NR>;
  constexpr int kChunks = D / 8;   // 16-byte pieces a row
  extern __shared__ __align__(1024) uint8_t win_smem[];
  __shared__ WinBars<C::kStages> B;
  __shared__ long long sum_s[C::kThreads / 32];
  __shared__ __align__(16) float row_s[C::kRows][4];  // maxima, or sums, of each row by warp
  __shared__ __align__(16) uint16_t use_s[2][8];  // by turns: a warp may be one tile ahead
  __shared__ uint8_t tok_s[C::kRows];  // the token of each row
  __shared__ __align__(4) uint16_t mask_s[C::kWarps][8 * C::kNR];  // keys of a warp's 16 that each row sees
  __shared__ int last_s;
  const AttnArgs &a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int groups = a.V, rows = a.kv.per * a.G;
  const uint32_t smem0 = smem_u32(win_smem);
  pdl_release();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 33);  // the producer's expected bytes, and its lanes' copies of queries
      mbar_init(&B.empty[i], C::kWarps);
    }
    B.abort = 0;
    mbar_fence_init();
  }

  for (int i = threadIdx.x; i < C::kRows; i += C::kThreads) tok_s[i] = (uint8_t)min(i / a.G, 255);

  pdl_wait();

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
  const int shares = (int)min((long long)gridDim.x, total), share = blockIdx.x;
  if (share >= shares) return;

  if (warp == C::kWarps) {
    // ---- producer: all but the pieces is uniform over the warp ----
    // lane l < pieces has piece l of a tile: a page, or half of one of 128
    const int log_pc = min(a.kv.log_ps, C::kLogBK), pc = 1 << log_pc, pieces = C::kBK >> log_pc;
    int st = 0, qn = 0, b = 0;
    uint32_t ph = 1;
    long long issued = 0, line = 0;  // line: tiles before sequence b
    const long long x0 = mul_div(total, share, shares);
    // the sequence of x0
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
    // (beyond the sequences, here or below, only where the lengths change under the call: no more tiles then)
    long long x1 = b < a.kv.n_seqs ? mul_div(total, share + 1, shares) : x0;
    b = min(b, a.kv.n_seqs - 1);
    SeqView s = seq_view(nullptr, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
    TileRange r = window_tiles(a, s, C::kLogBK);
    const int gi = x1 > x0 ? (int)mul_div(x0 - line, 1, r.count) : 0;
    int t = x1 > x0 ? (int)(x0 - line - (long long)gi * r.count) : 0;
    int hv = gi;
    // this lane's piece of the tile at the cursor
    auto piece = [&](bool &seen) {
      const int a0 = (tile_of(r, t) << C::kLogBK) + (lane << log_pc), e0 = a0 + pc;
      seen = lane < pieces && a0 < s.n && (a.window <= 0 || e0 - 1 > s.n - s.m - a.window || a0 < a.n_sinks);
      return seen ? __ldg(a.kv.table + (size_t)b * a.kv.max_pages + (a0 >> a.kv.log_ps)) : 0;
    };
    bool seen;
    int page = piece(seen);
    for (long long x = x0; x < x1; ++x) {
      if (!__all_sync(0xffffffffu, win_wait(&B.empty[st], ph, B, a.status))) break;
      const bool ok = seen && page >= 0 && page < a.kv.n_pages;
      const uint32_t good = __ballot_sync(0xffffffffu, ok), wrong = __ballot_sync(0xffffffffu, seen && !ok);
      const bool first = x == x0 || t == 0;
      const int j0 = tile_of(r, t) << C::kLogBK, cb = b, chv = hv;
      // below 2^31: checked on the host
      const int row = ((page * a.V + hv) << a.kv.log_ps) + ((j0 + (lane << log_pc)) & ((1 << a.kv.log_ps) - 1));
      if (lane == 0) {
        TileRec &rec = B.rec[st];
        const bool last = x + 1 == x1 || t + 1 == r.count;
        rec.b = b;
        rec.hv = hv;
        rec.j0 = j0;
        rec.n = s.n;
        rec.q = qn;
        rec.flags = (first ? kRecFirst : 0) | (last ? kRecLast : 0) |
                    (wrong || !tile_full(s.n - s.m, s.n - 1, j0, C::kBK, s.n, a.window, a.n_sinks) ? kRecPartial : 0);
        if (last) {
          const long long gs = x - t, ge = gs + r.count;
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
      // one elected lane issues all, on values that are uniform over the warp
      constexpr int kPieces = C::kBK / 16;
      int y[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) y[i] = __shfl_sync(0xffffffffu, row, i);
      if (elect_one()) {
        uint8_t *dst = win_smem + st * C::kStageBytes;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (good >> i & 1) {
            uint8_t *d = dst + i * pc * 128;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              tma_load_2d(d + h * C::kHalfBytes, &kmap, h * 64, y[i], &B.full[st]);
              tma_load_2d(d + C::kTileBytes + h * C::kHalfBytes, &vmap, h * 64, y[i], &B.full[st]);
            }
          }
      }
      __syncwarp();
      // the cursor, and the next tile's pages, which come in while this warp waits for a stage
      if (++t == r.count) {
        t = 0;
        if (++hv == a.V) {
          hv = 0;
          if (b + 1 == a.kv.n_seqs) x1 = x + 1;
          if (x + 1 < x1) {
            s = seq_view(nullptr, a.kv.kv_len, ++b, a.kv.per, a.T, a.kv.cap);
            r = window_tiles(a, s, C::kLogBK);
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
          const int rr = i / kChunks, ch = i % kChunks, tok = tok_s[rr];
          const bool in = rr < rows;
          const uint16_t *src = a.q + (in ? (size_t)(cb * a.kv.per + tok) * a.ld_q + (size_t)(chv * a.G + rr - tok * a.G) * D + ch * 8 : 0);
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

  // ---- the other warps: quarter wq of the keys and columns, rows rb on ----
  const int wq = warp & 3, rb = (warp >> 2) * 8 * C::kNR;
  constexpr int kMeet = C::kWarps * 32;
  uint32_t phase = 0;
  int cs = 0, turn = 0;
  uint32_t qf[C::kNR][D / 16][2];
  float o[C::kMD][C::kNR][4], m[C::kNR][2], l[C::kNR][2];  // columns of the C fragment: rows 8 i + 2 c and one more
  uint32_t qs = 0;                             // where the group's queries lie
  // lane offsets in a stage: 16 keys x 2 pieces of K for ldmatrix, 16 keys x 2 pieces of V for its transposed form
  const int kr = 16 * C::kMK * wq + (lane & 15), vr = (lane & 7) + ((lane >> 4) << 3);
  const uint32_t koff = (uint32_t)(kr * 128 + (((lane >> 4) ^ (kr & 7)) << 4));
  const uint32_t voff = (uint32_t)(C::kTileBytes + vr * 128);
  for (;;) {
    const bool came = win_wait(&B.full[cs], phase, B, a.status);
    const TileRec &rec = B.rec[cs];
    const int flags = came ? rec.flags : kRecEnd;
    const uint32_t st = smem0 + (uint32_t)cs * C::kStageBytes, ps = smem0 + C::kPAt + (uint32_t)turn * C::kPBytes;
    float sc[C::kMK][C::kNR][4];  // keys g and g + 8 of a tile, rows 2 c and 2 c + 1
    bool grow = flags & kRecEnd;
    if (!grow) {
      if (flags & kRecFirst) {
        qs = smem0 + C::kQAt + (uint32_t)rec.q * C::kQBytes;
#pragma unroll
        for (int i = 0; i < C::kNR; ++i) {
#pragma unroll
          for (int t = 0; t < C::kMD; ++t) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
          m[i][0] = m[i][1] = -INFINITY;
          l[i][0] = l[i][1] = 0.f;
          const int r = rb + 8 * i + (lane & 7);
#pragma unroll
          for (int k = 0; k < D / 16; k += 2)
            ldsm_x4(qs + (uint32_t)(r * kChunks + ((2 * k + (lane >> 3)) ^ (r & 7))) * 16u, qf[i][k][0], qf[i][k][1],
                    qf[i][k + 1][0], qf[i][k + 1][1]);
        }
      }
      // ---- scores of this warp's keys
#pragma unroll
      for (int t = 0; t < C::kMK; ++t) {
#pragma unroll
        for (int i = 0; i < C::kNR; ++i) sc[t][i][0] = sc[t][i][1] = sc[t][i][2] = sc[t][i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
          uint32_t kf[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            ldsm_x4((st + koff + (uint32_t)(t * 2048 + ((k + e) >> 2) * C::kHalfBytes)) ^ (uint32_t)(((k + e) & 3) << 5),
                    kf[e][0], kf[e][1], kf[e][2], kf[e][3]);
#pragma unroll
          for (int i = 0; i < C::kNR; ++i) {
            mma_bf16_16816(sc[t][i], kf[0], qf[i][k][0], qf[i][k][1], sc[t][i]);
            mma_bf16_16816(sc[t][i], kf[1], qf[i][k + 1][0], qf[i][k + 1][1], sc[t][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < C::kNR; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][i][e] *= a.scale_log2;
      }
      if (flags & kRecPartial) {
        // which of the warp's keys some row sees, and of these the ones whose values are not finite: 0 * v is NaN
        // then, so that where rows differ in what they see such a key is left out of the product, and the rows that
        // see it become NaN
        const int n = rec.n, j0 = rec.j0, base_pos = n - a.kv.per;
#pragma unroll
        for (int t = 0; t < C::kMK; ++t) {
          // lane and lane + 16 look at one key, half of its values each
          const int k0 = 16 * (C::kMK * wq + t), kk = k0 + (lane & 15), j = j0 + kk;
          const bool live = j < n && (a.window <= 0 || base_pos - j < a.window || j < a.n_sinks) &&
                            !(rec.bad[kk >> 5] >> (kk & 31) & 1);
          bool bad = false;
          if (live && a.kv.per > 1) {
            const uint8_t *v = win_smem + cs * C::kStageBytes + C::kTileBytes + kk * 128;
#pragma unroll
            for (int i = 0; i < kChunks / 2; ++i) {
              const int ch = (lane >> 4) * (kChunks / 2) + i;
              bad |= not_finite8(*reinterpret_cast<const uint4 *>(v + (ch >> 3) * C::kHalfBytes + (((ch & 7) ^ (kk & 7)) << 4)));
            }
          }
          const uint32_t lv = __ballot_sync(0xffffffffu, live) & 0xffffu;
          uint32_t bd = __ballot_sync(0xffffffffu, bad);
          bd = (bd | bd >> 16) & 0xffffu;
          if (lane == 0 && warp < 4) use_s[turn][C::kMK * wq + t] = (uint16_t)(lv & ~bd);
#pragma unroll
          for (int r = lane; r < 8 * C::kNR; r += 32) {
            const int hi = rb + r < rows ? base_pos + tok_s[rb + r] - (j0 + k0) : -1;  // keys up to hi,
            const int lo = a.window > 0 ? hi - a.window + 1 : 0;                       // from lo on
            const int sk = a.window > 0 ? a.n_sinks - (j0 + k0) : 0;                   // or below sk
            mask_s[warp][r] = (uint16_t)(below(hi + 1) & (~below(lo) | below(sk)) & lv);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::kNR; ++i) {
            // two rows' masks: this lane's keys are bits 0 and 8 of each after the shift
            const uint32_t both = *reinterpret_cast<const uint32_t *>(&mask_s[warp][8 * i + 2 * c]), v = both >> g;
            if (!(v & 1u)) sc[t][i][0] = -INFINITY;
            if (!(v & 0x10000u)) sc[t][i][1] = -INFINITY;
            if (!(v & 0x100u)) sc[t][i][2] = -INFINITY;
            if (!(v & 0x1000000u)) sc[t][i][3] = -INFINITY;
            if (bd) {
              if (both & bd) l[i][0] = NAN;
              if (both >> 16 & bd) l[i][1] = NAN;
            }
          }
          __syncwarp();
        }
      }
    }
    // ---- weights, with the maximum as it stands; once more when one has to grow.  (A loop, so that its code is there
    // once: a group's first tile always goes round twice.)
    float sums[C::kNR][2];
    bool grown = false, out = false;
    for (;;) {
      if (!(flags & kRecEnd)) {
#pragma unroll
        for (int i = 0; i < C::kNR; ++i) {
          if (grown) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 x = *reinterpret_cast<const float4 *>(&row_s[rb + 8 * i + 2 * c + e][0]);
              const float nm = fmaxf(m[i][e], fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
              const float f = ex2(m[i][e] - (nm == -INFINITY ? 0.f : nm));
              m[i][e] = nm;
              l[i][e] *= f;
#pragma unroll
              for (int t = 0; t < C::kMD; ++t) {
                o[t][i][e] *= f;
                o[t][i][2 + e] *= f;
              }
            }
          }
          // nothing seen yet: 2^(-inf - 0) = 0
          const float s0 = m[i][0] == -INFINITY ? 0.f : m[i][0], s1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
          const float most0 = m[i][0] + kWinLazy, most1 = m[i][1] + kWinLazy;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int t = 0; t < C::kMK; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = sc[t][i][2 * h], y = sc[t][i][2 * h + 1];
              grow |= !(x <= most0) || !(y <= most1);
              const float e0 = ex2(x - s0), e1 = ex2(y - s1);
              sum0 += e0;
              sum1 += e1;
              const int key = 16 * (C::kMK * wq + t) + g + 8 * h;
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(ps + (uint32_t)(((rb >> 3) + i) * (C::kBK * 16) + key * 16 + 4 * c)),
                           "r"(pack_bf16x2(e0, e1))
                           : "memory");
            }
          sums[i][0] = sum0;
          sums[i][1] = sum1;
        }
      }
      // the meeting: the weights are there, unless a maximum has to grow (or the end has come)
      const bool again = win_meet(grow && !grown, kMeet);
      if (!again) break;
      out = win_meet(!came, kMeet) || (flags & kRecEnd);  // all leave together when a wait has given up
      if (out) break;
#pragma unroll
      for (int i = 0; i < C::kNR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][i][e], sc[0][i][2 + e]);
          if constexpr (C::kMK == 2) x = fmaxf(x, fmaxf(sc[C::kMK - 1][i][e], sc[C::kMK - 1][i][2 + e]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          if (g == 0) row_s[rb + 8 * i + 2 * c + e][wq] = x;
        }
      win_meet(false, kMeet);
      grown = true;
    }
    if (out) break;
#pragma unroll
    for (int i = 0; i < C::kNR; ++i) {
      l[i][0] += sums[i][0];
      l[i][1] += sums[i][1];
    }
    // ---- products over this warp's columns, two 16-key steps a round
#pragma unroll
    for (int k = 0; k < C::kBK / 16; k += 2) {
      uint32_t vf[2][C::kMD][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < C::kMD; ++t) {
          const int ch = 2 * (C::kMD * wq + t) + ((lane >> 3) & 1);
          ldsm_x4_t(st + voff + (uint32_t)((k + e) * 2048 + (ch >> 3) * C::kHalfBytes + (((ch & 7) ^ (vr & 7)) << 4)),
                    vf[e][t][0], vf[e][t][1], vf[e][t][2], vf[e][t][3]);
        }
      if (flags & kRecPartial) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // this lane's keys of the two halves of a fragment: 2c, 2c + 1 and 8 more
          const uint32_t u = (uint32_t) * reinterpret_cast<const volatile uint16_t *>(&use_s[turn][k + e]) >> (2 * c);
          const uint32_t v0 = (u & 1 ? 0xffffu : 0u) | (u & 2 ? 0xffff0000u : 0u);
          const uint32_t v1 = (u & 256 ? 0xffffu : 0u) | (u & 512 ? 0xffff0000u : 0u);
#pragma unroll
          for (int t = 0; t < C::kMD; ++t) {
            vf[e][t][0] &= v0;
            vf[e][t][1] &= v0;
            vf[e][t][2] &= v1;
            vf[e][t][3] &= v1;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < C::kNR; ++i) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(ps + (uint32_t)(((rb >> 3) + i) * (C::kBK * 16) + (16 * k + lane) * 16), b0, b1, b2, b3);
#pragma unroll
        for (int t = 0; t < C::kMD; ++t) {
          mma_bf16_16816(o[t][i], vf[0][t], b0, b1, o[t][i]);
          mma_bf16_16816(o[t][i], vf[1][t], b2, b3, o[t][i]);
        }
      }
    }
    turn ^= 1;
    int c0 = 0, c1 = 0, slot = 0, slot0 = 0, hv = 0, q0 = 0;
    if (flags & kRecLast) {
      c0 = rec.c0;
      c1 = rec.c1;
      slot = rec.slot;
      slot0 = rec.slot0;
      hv = rec.hv;
      q0 = rec.b * a.kv.per;
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
    for (int i = 0; i < C::kNR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[i][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (g == 0) row_s[rb + 8 * i + 2 * c + e][wq] = x;
      }
    win_meet(false, kMeet);
    const int live = rows;
    constexpr size_t kPart = (size_t)C::kRows * (D + 2);
    float *po = a.part + ((size_t)share * 2 + slot) * kPart, *pm = po + (size_t)C::kRows * D;
#pragma unroll
    for (int i = 0; i < C::kNR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rb + 8 * i + 2 * c + e, col = 16 * C::kMD * wq + g;
        if (r >= live) continue;
        const float4 x = *reinterpret_cast<const float4 *>(&row_s[r][0]);
        const float sum = (x.x + x.y) + (x.z + x.w);
        if (c0 == c1) {
          const float inv = sum == 0.f ? 0.f : 1.0f / sum;
          const int tok = tok_s[r];
          uint16_t *dst = a.out + ((size_t)(q0 + tok) * a.H + (size_t)hv * a.G + r - tok * a.G) * D + col;
#pragma unroll
          for (int t = 0; t < C::kMD; ++t) {
            dst[16 * t] = float_to_bf16_bits(o[t][i][e] * inv);
            dst[16 * t + 8] = float_to_bf16_bits(o[t][i][2 + e] * inv);
          }
        } else {
#pragma unroll
          for (int t = 0; t < C::kMD; ++t) {
            __stcg(po + (size_t)r * D + col + 16 * t, o[t][i][e]);
            __stcg(po + (size_t)r * D + col + 16 * t + 8, o[t][i][2 + e]);
          }
          if (wq == 0 && g == 0) __stcg(reinterpret_cast<float2 *>(pm + 2 * r), make_float2(m[i][e], sum));
        }
      }
    if (c0 == c1 || w.join_after) continue;
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
    // two pieces of four columns a thread, with up to eight parts of both in flight
    for (int i0 = threadIdx.x; i0 < live * (D / 4); i0 += 2 * kMeet) {
      float mm[2] = {-INFINITY, -INFINITY}, ll[2] = {0.f, 0.f}, y[2][4] = {};
#pragma unroll 1
      for (int e0 = c0; e0 <= c1; e0 += 8) {
        float2 ml[2][8];
        float4 v[2][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = min(e0 + e, c1);  // behind the last one, the last with no weight
          const float *pk = a.part + ((size_t)k * 2 + (k == c0 ? slot0 : 0)) * kPart;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = min(i0 + u * kMeet, live * (D / 4) - 1);
            ml[u][e] = __ldcg(reinterpret_cast<const float2 *>(pk + (size_t)C::kRows * D + 2 * (i / (D / 4))));
            v[u][e] = __ldcg(reinterpret_cast<const float4 *>(pk + 4 * (size_t)i));
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float nm = mm[u];
#pragma unroll
          for (int e = 0; e < 8; ++e) nm = fmaxf(nm, ml[u][e].x);
          const float sub = nm == -INFINITY ? 0.f : nm, f0 = ex2(mm[u] - sub);
          mm[u] = nm;
          ll[u] *= f0;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[u][k] *= f0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e0 + e > c1) continue;
            const float f = ex2(ml[u][e].x - sub);
            ll[u] += ml[u][e].y * f;
            y[u][0] += v[u][e].x * f;
            y[u][1] += v[u][e].y * f;
            y[u][2] += v[u][e].z * f;
            y[u][3] += v[u][e].w * f;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + u * kMeet;
        if (i >= live * (D / 4)) continue;
        const float inv = ll[u] == 0.f ? 0.f : 1.0f / ll[u];
        const int rg = i / (D / 4), tok = tok_s[rg];
        uint16_t *dst = a.out + ((size_t)(q0 + tok) * a.H + (size_t)hv * a.G + rg - tok * a.G) * D + 4 * (i % (D / 4));
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16x2(y[u][0] * inv, y[u][1] * inv), pack_bf16x2(y[u][2] * inv, y[u][3] * inv));
      }
    }
  }
}

// The parts of one row of a cut group, in share order: threads are D/4 pieces of four columns times kLanes, which take
// every kLanes-th part each and are then summed in order.
template <int D>
__global__ void __launch_bounds__(512) attn_join_kernel(const __grid_constant__ WinArgs w, int tile_rows, int log_bk, int ctas) {
  constexpr int kQuads = D / 4, kLanes = 512 / kQuads;
  __shared__ float2 ml_s[kLanes];
  __shared__ float4 o_s[kLanes][kQuads];
  __shared__ long long total_s[17];
  const AttnArgs &a = w.a;
  const int groups = a.V, rows = a.kv.per * a.G;
  const int r = blockIdx.x % tile_rows, hv = blockIdx.x / tile_rows % groups, b = blockIdx.x / tile_rows / groups;
  pdl_release();
  pdl_wait();
  if (r >= rows) return;
  // the line, and where this sequence stands in it
  long long total = 0, line = 0;
  for (int i = threadIdx.x; i < a.kv.n_seqs; i += 512) {
    const int c = window_count(a, i, log_bk);
    total += c;
    if (i < b) line += c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    line += __shfl_xor_sync(0xffffffffu, line, o);
  }
  __shared__ long long line_s[16];
  if ((threadIdx.x & 31) == 0) {
    total_s[threadIdx.x >> 5] = total;
    line_s[threadIdx.x >> 5] = line;
  }
  __syncthreads();
  total = line = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    total += total_s[i];
    line += line_s[i];
  }
  total *= groups;
  const int count = window_count(a, b, log_bk), shares = (int)min((long long)ctas, total);
  const long long gs = line * groups + (long long)hv * count, ge = gs + count;
  const int c0 = share_of(gs, shares, total), c1 = share_of(ge - 1, shares, total);
  if (c0 == c1) return;  // not cut
  const int slot0 = gs > mul_div(total, c0, shares);
  const size_t part = (size_t)tile_rows * (D + 2);
  const int q = threadIdx.x % kQuads, lane = threadIdx.x / kQuads;
  float m = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k0 = c0 + lane; k0 <= c1; k0 += 8 * kLanes) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = min(k0 + e * kLanes, c1);  // behind the last one, the last with no weight
      const float *p = a.part + ((size_t)k * 2 + (k == c0 ? slot0 : 0)) * part;
      ml[e] = __ldcg(reinterpret_cast<const float2 *>(p + (size_t)tile_rows * D + 2 * r));
      v[e] = __ldcg(reinterpret_cast<const float4 *>(p + (size_t)r * D) + q);
    }
    float nm = m;
#pragma unroll
    for (int e = 0; e < 8; ++e) nm = fmaxf(nm, ml[e].x);
    const float sub = nm == -INFINITY ? 0.f : nm, f0 = ex2(m - sub);
    m = nm;
    l *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] *= f0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (k0 + e * kLanes > c1) continue;
      const float f = ex2(ml[e].x - sub);
      l += ml[e].y * f;
      y[0] += v[e].x * f;
      y[1] += v[e].y * f;
      y[2] += v[e].z * f;
      y[3] += v[e].w * f;
    }
  }
  if (q == 0) ml_s[lane] = make_float2(m, l);
  o_s[lane][q] = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (lane != 0) return;
  float mm = -INFINITY, ll = 0.f, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kLanes; ++i) mm = fmaxf(mm, ml_s[i].x);
  const float sub = mm == -INFINITY ? 0.f : mm;
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const float f = ex2(ml_s[i].x - sub);
    const float4 v = o_s[i][q];
    ll += ml_s[i].y * f;
    z[0] += v.x * f;
    z[1] += v.y * f;
    z[2] += v.z * f;
    z[3] += v.w * f;
  }
  const float inv = ll == 0.f ? 0.f : 1.0f / ll;
  const int tok = r / a.G;
  uint16_t *dst = a.out + ((size_t)(b * a.kv.per + tok) * a.H + (size_t)hv * a.G + r - tok * a.G) * D + 4 * q;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(z[0] * inv, z[1] * inv), pack_bf16x2(z[2] * inv, z[3] * inv));
}

template <int D, int NR>
cudaError_t launch(WinArgs w, const moe_kv_cache &c, cudaStream_t s) {
  using C = WinCfg<D, NR>;
  CUtensorMap km, vm;
  if (!make_pages_map(&km, c.k, c.n_pages, w.a, D, C::kBK) || !make_pages_map(&vm, c.v, c.n_pages, w.a, D, C::kBK))
    return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(attn_window_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  // more than kJoinParts parts a group, were all sequences alike: the second launch
  const int ctas = kAttnSms * C::kCtas;
  const long long groups = (long long)w.a.kv.n_seqs * w.a.V;
  w.join_after = groups * kJoinParts < ctas && w.a.kv.cap > kJoinParts * C::kBK;
  err = launch_dependent(attn_window_kernel<D, NR>, ctas, C::kThreads, C::kSmem, 1, s, km, vm, w);
  if (err == cudaSuccess && w.join_after)
    err = launch_dependent(attn_join_kernel<D>, (unsigned)groups * C::kRows, 512, 0, 1, s, w, C::kRows, C::kLogBK, ctas);
  return err;
}

// Rows of a window: one, two or four 8-row tiles side by side.
template <int D>
cudaError_t launch_d(const WinArgs &w, const moe_kv_cache &c, cudaStream_t s) {
  const int rows = w.a.kv.per * w.a.G;
  return rows <= 8    ? launch<D, 1>(w, c, s)
         : rows <= 16 ? launch<D, 2>(w, c, s)
                      : launch<D, 4>(w, c, s);
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
  // of windows two parts a share (with more than 16 rows, one CTA a SM, there are half as many shares); of chunks one a
  // CTA that shares an item, of which there are at most kAttnSms, with its rows' maxima and sums and the items' rows
  const size_t windows = (size_t)kAttnShares * 2 * (8 * d.n_heads / d.n_kv_heads <= 8 ? 8 : 16) * (d.head_dim + 2) * 4;
  return std::max(windows, (size_t)kAttnSms * (256 * (d.head_dim * 4 + 8) + 8));
}

cudaError_t launch_attn(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s) {
  const WinArgs w{a, 0};
  trace_mark(MOE_KERNEL_ATTN, false, s);
  const int rows = a.kv.per * a.G;
  const bool few = rows > 16 && (long long)a.kv.n_seqs * a.V <= kWinFew;
  const bool window = !a.kv.q_start && a.kv.per <= 8 && rows <= kWinRows && !few;
  const cudaError_t err = !window             ? launch_attn_tc(d, a, c, s)
                          : d.head_dim == 128 ? launch_d<128>(w, c, s)
                                              : launch_d<64>(w, c, s);
  trace_mark(MOE_KERNEL_ATTN, true, s);
  return err;
}

}  // namespace moe
