// Attention of prompt chunks over the paged cache on the 5th-generation tensor cores (tcgen05, sm_100a).
//
// A CTA takes one key/value head of one sequence and up to two tiles of 128 rows; a tile's rows are (token, head of
// the group) pairs, so that all heads of a group share the keys that were loaded for one.  It walks the 128-key
// tiles that its rows see.  For each of its row tiles i and key tile j, with the softmax's running maximum m and sum l:
//   S_i = Q_i K_j^T            (tensor memory, fp32)
//   P_i = 2^(scale S_i - m)    (one thread a row; bf16, over S_i in tensor memory)
//   O_i += P_i V_j             (tensor memory, fp32)
// The products of one row tile run under the softmax of the other.  A tile's chain of softmax (2300 cycles), P V and the
// next Q K (700 and 620) paces it: 8192 tokens of 16 heads over 2 key/value heads take 252 us from idle, 1095 TFLOP/s (281
// and 980 in calls one behind another, at the clock that the power limit leaves), with the tensor core busy half of the
// time.  Slower, from idle too: two threads a row (309 us, the exchange of the halves' maxima), a
// quarter or half of the exponentials as polynomials on the FMA units (264, 302: the special function unit is not the
// limit), weights begun before the maximum is known (262), steps of 64 keys with two places for S, so that the next Q K
// runs under the softmax (394: 64 columns take the tensor core as long as 128).  m is the maximum seen so far, left as it is
// until a row exceeds it by 8 (a factor of 256, which fp32 sums and bf16 weights carry without loss: only then are l
// and O_i, which lie in tensor memory, rescaled), so that the rescaling is rare.
//   warps 0-3, 4-7 : softmax of row tile 0, 1, then its output rows;
//   warp 8         : TMA: queries once, K and V a page at a time, into rings of 128-key stages;
//   warp 9         : tcgen05.mma issue;
//   warps 10, 11   : V rows that must not be multiplied (keys that no row sees, non-finite values behind a mask)
//                    are cleared before P V, in tiles with a mask only.
// Few row tiles over many keys leave SMs idle: then a cluster of 2, 4 or 8 CTAs shares the key tiles of one pair of row
// tiles.  Each finishes its part of the rows from all of their (m, l, O), in rank order.  Where clusters, which are powers
// of two and find no room beyond 14 of 8, would leave too many idle, parts in any number are joined by a second launch.
// 1024 tokens alone take 21 us (2 CTAs a pair), 16 tokens on 32768 19 us (74 parts a key/value head).
// Every wait on memory is bounded (sync.cuh).
#include <algorithm>

#include "attn.cuh"
#include "half.cuh"

namespace moe {
namespace {

constexpr int kTcBK = 128;   // keys a tile
constexpr int kTcLogBK = 7;
constexpr int kTcRows = 128;
constexpr int kTcThreads = 384;
constexpr int kTcInfo = 8;   // ring of tile descriptions: more than the tiles between the producer and a softmax
constexpr float kTcLazy = 8.0f;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // of a thread: 256 x 216 + 128 x 72 are the launch's 384 x 168

template <int D>
struct TcCfg {
  static constexpr int kHalves = D / 64;                    // 64-column halves of a row (one swizzle row each)
  static constexpr int kHalfBytes = 128 * 128;              // 128 rows x 64 columns
  static constexpr int kTileBytes = kHalves * kHalfBytes;   // a Q, K or V tile
  static constexpr int kStages = 2;                         // K and V stages each
  static constexpr int kSmemTiles = 2 + 2 * kStages;
  static constexpr uint32_t kS = 0, kO = 256;               // tensor memory columns: S0 S1, O0 O1
  static constexpr uint32_t kTmemCols = 512;
};

struct TileInfo {
  int partial;       // some row does not see some key of the tile
  uint32_t bad[4];   // keys whose page is outside the cache
};

template <int D>
struct TcBars {
  uint64_t q_full, k_full[TcCfg<D>::kStages], k_empty[TcCfg<D>::kStages], v_full[TcCfg<D>::kStages],
      v_ready[TcCfg<D>::kStages], v_empty[TcCfg<D>::kStages], s_full[2], p_ready[2][2], pv_done[2], done;
  TileInfo info[kTcInfo];
  uint32_t flagged[TcCfg<D>::kStages][4];  // keys of a V stage whose values are not finite
  uint32_t tmem;
  int abort;
  uint8_t tok[128];  // token of each row of a tile, w.tokens for the rows behind the last
  float2 ml[256];  // maximum and sum of each row, for the other CTAs of a cluster
  int found_b, found_t, warp_sum[kTcThreads / 32];
};

struct TcArgs {
  AttnArgs a;
  int tokens;  // tokens a row tile: 128 / G
  int log_splits;  // log2 of the CTAs of a cluster, which share an item's key tiles
  int parts;       // else the CTAs that share them without a cluster, joined by a second launch; or 0
  float2 *ml;      // [CTAs, 256] maximum and sum of each row of the parts
  int2 *rows;      // [items x V] first row and number of tokens of an item
};

template <class Bars>
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity, Bars &B, uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int *>(&B.abort)) return false;
  if (!mbar_wait(bar, parity)) {
    set_status(status, kStatusTimeout);
    B.abort = 1;
    return false;
  }
  return true;
}

// B operand with N contiguous (V: keys x head_dim): 64-column groups kHalfBytes apart, 8-key groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_n_sw128(uint32_t addr, uint32_t group_bytes) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(group_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Where the rows of a pair of row tiles go.
struct TcRows {
  uint16_t *out;  // of the sequence's first new token and the group's first head
  int H, G, tok0, tokens, m, nq;
};

// The rows of one CTA of a cluster of 2^LS: row own * split + k for k = first, first + step, ..., all parts of all rows
// of a lane in flight at once.  `mine`: this CTA's part in shared memory; `parts`: the others', in the same layout.
template <int D, int LS>
__device__ __forceinline__ void tc_join(const TcRows &w, const float2 *ml, const uint8_t *tok, const float *mine,
                                        const float *parts, int split, int first, int sub) {
  constexpr int kQuads = D / 4, kStep = 8 * (32 / kQuads), kOwn = 256 >> LS, kRows = kOwn / kStep, kParts = 1 << LS;
  const int own = w.nq * 128 >> LS;
  float4 o[kRows][kParts];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int q = own * split + min(first + u * kStep, own - 1), piece = (sub ^ (q & (kQuads - 1))) << 2;
#pragma unroll
    for (int p = 0; p < kParts; ++p)
      o[u][p] = p == split ? *reinterpret_cast<const float4 *>(mine + (size_t)q * D + piece)
                           : __ldcg(reinterpret_cast<const float4 *>(parts + ((size_t)p * 256 + q) * D + piece));
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int k = first + u * kStep, r = own * split + k, i = r >> 7, rt = tok[r & 127];
    const int tk = w.tok0 + i * w.tokens + rt;
    if (k >= own || rt >= w.tokens || tk >= w.m) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int p = 0; p < kParts; ++p) mx = fmaxf(mx, ml[p * kOwn + k].x);
    const float sub_m = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const float2 x = ml[p * kOwn + k];
      const float f = ex2(x.x - sub_m);
      sum += f * x.y;
      y[0] += f * o[u][p].x;
      y[1] += f * o[u][p].y;
      y[2] += f * o[u][p].z;
      y[3] += f * o[u][p].w;
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t *dst = w.out + ((size_t)tk * w.H + (r & 127) - rt * w.G) * D + sub * 4;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv));
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TcArgs w) {
  using C = TcCfg<D>;
  extern __shared__ __align__(1024) uint8_t tc_raw[];
  uint8_t *smem = tc_raw + ((1024u - (smem_u32(tc_raw) & 1023u)) & 1023u);
  uint8_t *q_s = smem, *k_s = smem + 2 * C::kTileBytes, *v_s = k_s + C::kStages * C::kTileBytes;
  TcBars<D> &B = *reinterpret_cast<TcBars<D> *>(smem + C::kSmemTiles * C::kTileBytes);
  const AttnArgs &a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = w.parts ? w.parts : 1 << w.log_splits;
  const int unit = w.parts ? blockIdx.x / w.parts : blockIdx.x >> w.log_splits, split = blockIdx.x - unit * splits;
  const int hv = unit % a.V, item = unit / a.V;
  pdl_release();
  // what needs no memory that others write
  if (threadIdx.x < 128) B.tok[threadIdx.x] = (uint8_t)min((int)threadIdx.x / a.G, w.tokens);
  if (threadIdx.x == 0) {
    mbar_init(&B.q_full, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.k_full[i], 1);
      mbar_init(&B.k_empty[i], 1);
      mbar_init(&B.v_full[i], 1);
      mbar_init(&B.v_ready[i], 2);
      mbar_init(&B.v_empty[i], 3);  // the products' commit and the two clearing warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_ready[i][0], 4);
      mbar_init(&B.p_ready[i][1], 4);
      mbar_init(&B.pv_done[i], 1);
    }
    mbar_init(&B.done, 1);
    B.abort = 0;
    mbar_fence_init();
    B.found_b = -1;
  }
  if (warp == 8 && lane < 3) tma_prefetch_map(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
  pdl_wait();
  // tensor memory only now: a launch that held it while it waits could keep it from one that it waits for

  // ---- which rows: items count row-tile pairs from the last sequence's last pair (with a causal mask the largest)
  if (blockIdx.x == 0) check_sequences(a.kv, a.T, a.status);
  __syncthreads();
  const int pair = 2 * w.tokens;
  int b, ft;
  if (!a.kv.q_start) {
    const int pairs = (a.kv.per + pair - 1) / pair, back = item / pairs;
    b = a.kv.n_seqs - 1 - back;
    ft = pairs - 1 - (item - back * pairs);
  } else {
    for (int c0 = 0, base = 0; c0 < a.kv.n_seqs; c0 += kTcThreads) {
      const int b = a.kv.n_seqs - 1 - (c0 + (int)threadIdx.x);
      const int cnt = b >= 0 ? (seq_view(a.kv.q_start, a.kv.kv_len, b, 0, a.T, a.kv.cap).m + pair - 1) / pair : 0;
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) B.warp_sum[warp] = incl;
      __syncthreads();
      int before = base, total = 0;
      for (int i = 0; i < kTcThreads / 32; ++i) {
        if (i < warp) before += B.warp_sum[i];
        total += B.warp_sum[i];
      }
      const int at = item - (before + incl - cnt);
      if (at >= 0 && at < cnt) {
        B.found_b = b;
        B.found_t = cnt - 1 - at;
      }
      base += total;
      __syncthreads();
      if (item < base) break;
    }
    b = B.found_b;
    ft = B.found_t;
  }
  if (b < 0) {
    if (w.parts && split == 0 && threadIdx.x == 0) w.rows[unit] = make_int2(0, 0);
    return;  // with the whole cluster, which has one item
  }
  // A CTA without key tiles comes to the join almost at once: before it writes the others' shared memory they have to
  // run, which it waits for there.
  const bool clustered = splits > 1 && !w.parts;
  if (clustered) cluster_started();
  const SeqView s = seq_view(a.kv.q_start, a.kv.kv_len, b, a.kv.per, a.T, a.kv.cap);
  const int tok0 = ft * pair;
  const int nq = s.m - tok0 > w.tokens ? 2 : 1;
  const int base = s.n - s.m;
  const int p0 = base + tok0, p1 = base + min(s.m, tok0 + pair) - 1;
  const TileRange tr = tile_range(p0, p1, s.n, a.window, a.n_sinks, kTcLogBK);
  // this CTA's key tiles: t0 .. t0 + nt - 1 of the range
  int tile0, nt;
  if (w.parts) {  // count x parts stays below 2^31: positions are below 2^30
    tile0 = tr.count * split / w.parts;
    nt = tr.count * (split + 1) / w.parts - tile0;
    if (split == 0 && threadIdx.x == 0) w.rows[unit] = make_int2(s.q0 + tok0, min(s.m - tok0, pair));
  } else {
    tile0 = (int)((long long)tr.count * split >> w.log_splits);
    nt = (int)((long long)tr.count * (split + 1) >> w.log_splits) - tile0;
  }
  const int32_t *table = a.kv.table + (size_t)b * a.kv.max_pages;

  if (warp == 9) tmem_alloc(&B.tmem, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = B.tmem;
  float m = -INFINITY, l = 0.f;  // of a row, in its softmax thread: m in units of log2, scaled

  // Registers go from the last four warps to the softmax.
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8) {
    // ---- producer ----
    const int rows = w.tokens * a.G;
    if (nt > 0 && elect_one()) {
      mbar_arrive_expect_tx(&B.q_full, (uint32_t)(nq * C::kHalves * rows * 128));
      for (int i = 0; i < nq; ++i)
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_3d(q_s + i * C::kTileBytes + h * C::kHalfBytes, &qmap, h * 64, hv * a.G, s.q0 + tok0 + i * w.tokens,
                      &B.q_full);
    }
    __syncwarp();
    const int ps = 1 << a.kv.log_ps, pages = kTcBK >> a.kv.log_ps;
    int issued_k = 0, issued_v = 0;
    for (int t = 0; t < nt; ++t) {
      const int st = t % C::kStages, j0 = tile_of(tr, tile0 + t) << kTcLogBK;
      const uint32_t ph = ((t / C::kStages) & 1) ^ 1;
      if (!__all_sync(0xffffffffu, at_wait(&B.k_empty[st], ph, B, a.status))) break;
      // lane l < pages: page l of the tile
      const int a0 = j0 + (lane << a.kv.log_ps), e0 = a0 + ps;
      const bool seen = lane < pages && a0 < s.n && a0 <= p1 &&
                        (a.window <= 0 || e0 - 1 > p0 - a.window || a0 < a.n_sinks);
      const int page = seen ? __ldg(table + (a0 >> a.kv.log_ps)) : 0;
      const bool ok = seen && page >= 0 && page < a.kv.n_pages;
      const uint32_t good = __ballot_sync(0xffffffffu, ok), wrong = __ballot_sync(0xffffffffu, seen && !ok);
      if (lane == 0) {
        TileInfo &in = B.info[t % kTcInfo];
        in.partial = wrong || !tile_full(p0, p1, j0, kTcBK, s.n, a.window, a.n_sinks);
        in.bad[0] = in.bad[1] = in.bad[2] = in.bad[3] = 0;
        if (wrong) {
          for (int k = 0; k < kTcBK; ++k)
            if (wrong >> (k >> a.kv.log_ps) & 1) in.bad[k >> 5] |= 1u << (k & 31);
          set_status(a.status, kStatusBadIndex);
        }
        mbar_arrive_expect_tx(&B.k_full[st], (uint32_t)(__popc(good) * ps * D * 2));
      }
      __syncwarp();
      const int row = (page * a.V + hv) << a.kv.log_ps;  // below 2^31: checked on the host
      if (ok)
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_2d(k_s + st * C::kTileBytes + h * C::kHalfBytes + lane * ps * 128, &kmap, h * 64, row, &B.k_full[st]);
      issued_k = t + 1;
      __syncwarp();
      if (!__all_sync(0xffffffffu, at_wait(&B.v_empty[st], ph, B, a.status))) break;
      if (lane == 0) mbar_arrive_expect_tx(&B.v_full[st], (uint32_t)(__popc(good) * ps * D * 2));
      __syncwarp();
      if (ok)
        for (int h = 0; h < C::kHalves; ++h)
          tma_load_2d(v_s + st * C::kTileBytes + h * C::kHalfBytes + lane * ps * 128, &vmap, h * 64, row, &B.v_full[st]);
      issued_v = t + 1;
      __syncwarp();
    }
    // every copy issued must land before the CTA exits, also after an abort
    if (nt > 0 && !mbar_wait(&B.q_full, 0)) set_status(a.status, kStatusTimeout);
    for (int t = max(0, issued_k - C::kStages); t < issued_k; ++t)
      if (!mbar_wait(&B.k_full[t % C::kStages], (t / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
    for (int t = max(0, issued_v - C::kStages); t < issued_v; ++t)
      if (!mbar_wait(&B.v_full[t % C::kStages], (t / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
  } else if (warp == 9) {
    // ---- products: the warp runs the loop on uniform values, one elected lane issues ----
    const uint32_t idesc_s = umma_idesc_bf16(kTcRows, kTcBK);
    const uint32_t idesc_o = umma_idesc_bf16(kTcRows, D) | (1u << 16);  // B with N contiguous
    auto scores = [&](int i, int t) {
      const uint32_t qa = smem_u32(q_s) + i * C::kTileBytes, ka = smem_u32(k_s) + (t % C::kStages) * C::kTileBytes;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * C::kHalfBytes + (k & 3) * 32;
          umma_ss(tbase + C::kS + i * kTcBK, umma_sdesc_sw128(qa + off), umma_sdesc_sw128(ka + off), idesc_s, k != 0);
        }
        umma_commit(&B.s_full[i]);
        if (i == nq - 1) umma_commit(&B.k_empty[t % C::kStages]);
      }
      __syncwarp();
    };
    if (nt > 0) {
      at_wait(&B.q_full, 0, B, a.status);
      at_wait(&B.k_full[0], 0, B, a.status);
      tc_fence_after();
      for (int i = 0; i < nq; ++i) scores(i, 0);
    }
    for (int t = 0; t < nt; ++t) {
      const int st = t % C::kStages;
      const uint32_t ph = (t / C::kStages) & 1;
      for (int i = 0; i < nq; ++i) {
        const uint32_t va = smem_u32(v_s) + st * C::kTileBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the weights of the first 64 keys, then the others'
          at_wait(&B.p_ready[i][h], t & 1, B, a.status);
          if (i == 0 && h == 0) {
            at_wait(&B.v_full[st], ph, B, a.status);
            at_wait(&B.v_ready[st], ph, B, a.status);
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              umma_ts(tbase + C::kO + i * D, tbase + C::kS + i * kTcBK + k * 8, sdesc_n_sw128(va + k * 2048, C::kHalfBytes),
                      idesc_o, (t | k) != 0);
            if (h == 1) {
              umma_commit(&B.pv_done[i]);
              if (i == nq - 1) umma_commit(&B.v_empty[st]);
            }
          }
          __syncwarp();
        }
        if (t + 1 < nt) {
          if (i == 0) at_wait(&B.k_full[(t + 1) % C::kStages], ((t + 1) / C::kStages) & 1, B, a.status);
          at_wait(&B.pv_done[i], t & 1, B, a.status);  // S_i(t + 1) goes over P_i(t)
          tc_fence_after();
          scores(i, t + 1);
        }
      }
    }
    if (elect_one()) {
      umma_commit(&B.done);
      if (!mbar_wait(&B.done, 0)) set_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else {
    // ---- V rows that must not be multiplied ----
    for (int t = 0; t < nt; ++t) {
      const int st = t % C::kStages, j0 = tile_of(tr, tile0 + t) << kTcLogBK;
      at_wait(&B.v_full[st], (t / C::kStages) & 1, B, a.status);
      const TileInfo &in = B.info[t % kTcInfo];
      if (in.partial) {
        uint8_t *v = v_s + st * C::kTileBytes;
        // lane and step pick a row: 32 rows a step and warp, each row by one lane
        for (int r0 = (warp - 10) * 32; r0 < kTcBK; r0 += 64) {
          const int r = r0 + lane, j = j0 + r;
          const bool live = j <= p1 && j < s.n && (a.window <= 0 || p0 - j < a.window || j < a.n_sinks) &&
                            !(in.bad[r >> 5] >> (r & 31) & 1);
          bool clear = !live;
#pragma unroll
          for (int i = 0; i < C::kHalves * 8; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(v + (i >> 3) * C::kHalfBytes + r * 128 + (((i & 7) + r) & 7) * 16);
            const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) clear |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
          }
          const uint32_t flag = __ballot_sync(0xffffffffu, live && clear);
          if (lane == 0) B.flagged[st][r0 >> 5] = flag;
          if (clear)
            for (int i = 0; i < C::kHalves * 8; ++i)
              *reinterpret_cast<uint4 *>(v + (i >> 3) * C::kHalfBytes + r * 128 + (((i & 7) + r) & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&B.v_ready[st]);
        mbar_arrive(&B.v_empty[st]);
      }
    }
  }
  if (splits > 1) {  // the meetings of the parts, below
    __syncthreads();
    if (clustered) {
      cluster_wait_started();
      cluster_meet();
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax of row tile i: one thread a row ----
    const int i = warp >> 2, row = threadIdx.x & 127;
    if (i < nq) {
      const int tok = tok0 + i * w.tokens + row / a.G;
      const bool alive = row < w.tokens * a.G && tok < s.m;
      const int pos = alive ? base + tok : -1;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t ts = tbase + lanes + C::kS + i * kTcBK, to = tbase + lanes + C::kO + i * D;
      const float scale = a.scale_log2;
      for (int t = 0; t < nt; ++t) {
        const int st = t % C::kStages, j0 = tile_of(tr, tile0 + t) << kTcLogBK;
        at_wait(&B.s_full[i], t & 1, B, a.status);
        tc_fence_after();
        const TileInfo &in = B.info[t % kTcInfo];
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
        tmem_wait_ld();
        uint32_t seen[4];
        if (in.partial) {
          // the keys of the tile that this row sees: columns up to hi, from lo on or below the sinks
          const int hi = min(pos, s.n - 1) - j0 + 1;
          const int lo = a.window > 0 ? pos - a.window + 1 - j0 : 0;
          const int sk = a.window > 0 ? a.n_sinks - j0 : 0;
          const float none = scale < 0.f ? INFINITY : -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            seen[k] = (below(lo - 32 * k) ^ 0xffffffffu | below(sk - 32 * k)) & below(hi - 32 * k) & ~in.bad[k];
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!(seen[c >> 5] >> (c & 31) & 1)) x[c] = none;
        }
        float mx;
        if (scale >= 0.f) {
          float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
          for (int c = 4; c + 7 < 128; c += 8) {
            m0 = max3_nan(m0, x[c], x[c + 1]);
            m1 = max3_nan(m1, x[c + 2], x[c + 3]);
            m2 = max3_nan(m2, x[c + 4], x[c + 5]);
            m3 = max3_nan(m3, x[c + 6], x[c + 7]);
          }
          m0 = max3_nan(m0, x[124], x[125]);
          m1 = max3_nan(m1, x[126], x[127]);
          mx = max3_nan(max3_nan(m0, m1, m2), m3, m3);
        } else {
          mx = x[0];
#pragma unroll
          for (int c = 1; c < 128; ++c) mx = min_nan(mx, x[c]);
        }
        mx *= scale;  // scale is not 0
        if (mx == INFINITY) mx = NAN;  // an infinite score that is seen: the whole row is NaN
        // a row that exceeds its maximum by more than the slack, or has none yet, takes the new one
        const bool grow = alive && !(mx <= m + kTcLazy);
        if (__any_sync(0xffffffffu, grow)) {
          const float nm = grow ? mx : m;
          const float f = m == -INFINITY ? 0.f : ex2(m - nm);  // l and O are 0 without a maximum
          if (t > 0) {
            at_wait(&B.pv_done[i], (t - 1) & 1, B, a.status);
            tc_fence_after();
            const float fo = grow ? f : 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t v[32];
              tmem_ld_32x32b_x16(to + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fo);
              tmem_st_32x32b_x16(to + c, v);
            }
            tmem_wait_st();
          }
          if (grow) {
            l *= f;
            m = nm;
          }
        }
        const float sub = m == -INFINITY ? 0.f : m;
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 64 * h; c < 64 * h + 64; c += 32) {
            uint32_t p[32];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float y0 = -sub, y1 = -sub, y2 = -sub, y3 = -sub;
              fma2(y0, y1, x[c + e], x[c + e + 1], scale, scale);
              fma2(y2, y3, x[c + e + 2], x[c + e + 3], scale, scale);
              y0 = ex2(y0);
              y1 = ex2(y1);
              y2 = ex2(y2);
              y3 = ex2(y3);
              add2(l0, l1, y0, y1);
              add2(l2, l3, y2, y3);
              p[e / 2] = pack_bf16x2(y0, y1);
              p[e / 2 + 1] = pack_bf16x2(y2, y3);
            }
            tmem_st_32x32b_x16(ts + c / 2, p);
          }
          if (h == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.p_ready[i][0]);
          }
        }
        l += (l0 + l1) + (l2 + l3);
        if (in.partial) {
          // a value that is not finite was left out of P V: rows that see it become NaN
          at_wait(&B.v_ready[st], (t / C::kStages) & 1, B, a.status);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (seen[k] & B.flagged[st][k]) l = NAN;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_ready[i][1]);
      }
      if (splits == 1) {
        // ---- output rows ----
        if (nt > 0) at_wait(&B.pv_done[i], (nt - 1) & 1, B, a.status);
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        // through the query tile's place (its products are done), so that a warp writes whole rows
        uint8_t *os = q_s + i * C::kTileBytes + row * (D * 2);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          if (nt > 0) {
            tmem_ld_32x32b_x32(to + c, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = nt > 0 && l != 0.f ? pack_bf16x2(__uint_as_float(v[e + 2 * k]) * inv, __uint_as_float(v[e + 2 * k + 1]) * inv) : 0u;
            *reinterpret_cast<uint4 *>(os + ((((c + e) >> 3) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        __syncwarp();
        constexpr int kPieces = D / 8, kRowsOnce = 32 / kPieces;
        const int wrow = 32 * (warp & 3);
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += kRowsOnce) {
          const int r = wrow + r0 + lane / kPieces, ch = lane % kPieces;
          const int rt = B.tok[r], tk = tok0 + i * w.tokens + rt;
          if (rt >= w.tokens || tk >= s.m) continue;
          const uint4 o = *reinterpret_cast<const uint4 *>(q_s + i * C::kTileBytes + r * (D * 2) + ((ch ^ (r & 7)) << 4));
          *reinterpret_cast<uint4 *>(a.out + ((size_t)(s.q0 + tk) * a.H + (size_t)hv * a.G + r - rt * a.G) * D + ch * 8) = o;
        }
      }
    }
    if (splits > 1) {
      // ---- the cluster's parts: O of this CTA's keys into the stages' place, rows of D fp32 in swizzled 16-byte
      // pieces.  A CTA finishes every splits-th part of the rows: it gets the others' (m, l) into its shared memory, and their rows by
      // way of the workspace in one asynchronous copy an owner (fetched through distributed shared memory 64 KB took
      // 7.5 us, stored to the workspace by the threads 2.3 us).  Parts without a cluster go there whole.
      constexpr int kQuads = D / 4;
      const int log_own = 6 + nq - w.log_splits, own = 1 << log_own;  // rows a CTA finishes: nq * 128 / splits
      __syncthreads();  // no product or copy needs the stages any more
      if (clustered) cluster_wait_started();
      if ((warp >> 2) < nq) {
        const int i = warp >> 2, row = threadIdx.x & 127, r = i * 128 + row;
        const uint32_t to = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + C::kO + i * D;
        float *os = reinterpret_cast<float *>(k_s) + (size_t)r * D;
        if (nt > 0) {
          at_wait(&B.pv_done[i], (nt - 1) & 1, B, a.status);
          tc_fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          if (nt > 0) {
            tmem_ld_32x32b_x32(to + c, v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4 *>(os + ((((c + e) >> 2) ^ (row & (kQuads - 1))) << 2)) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        if (w.parts) {
          __stcg(w.ml + (size_t)blockIdx.x * 256 + r, make_float2(m, l));
        } else {
          const int owner = r >> log_own, k = r & (own - 1);
          cluster_store2(cluster_map(smem_u32(&B.ml[(split << 8 >> w.log_splits) + k]), owner), m, l);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      named_bar(1, 256);
      constexpr int kRowsOnce = 32 / kQuads;
      const int sub = lane % kQuads, first = warp * kRowsOnce + lane / kQuads;
      float *parts = a.part + (size_t)(blockIdx.x - split) * 256 * D;  // of the item
      const float *mine = reinterpret_cast<const float *>(k_s);
      if (threadIdx.x < splits && (w.parts ? threadIdx.x == 0 && nt > 0 : (int)threadIdx.x != split)) {
        const int rows = w.parts ? nq * 128 : own, r = w.parts ? 0 : (int)threadIdx.x * own;
        bulk_store(parts + ((size_t)split * 256 + r) * D, smem_u32(mine + (size_t)r * D), (uint32_t)(rows * D * 4));
      }
      __syncwarp();
      if (clustered) cluster_meet();  // releases and acquires what went to the workspace too
      const TcRows where{a.out + ((size_t)s.q0 * a.H + (size_t)hv * a.G) * D, a.H, a.G, tok0, w.tokens, s.m, nq};
      if (w.parts)
        ;  // attn_tc_join_kernel
      else if (w.log_splits == 1)
        tc_join<D, 1>(where, B.ml, B.tok, mine, parts, split, first, sub);
      else if (w.log_splits == 2)
        tc_join<D, 2>(where, B.ml, B.tok, mine, parts, split, first, sub);
      else
        tc_join<D, 3>(where, B.ml, B.tok, mine, parts, split, first, sub);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// The parts of one row, in order: 8 warps take every 8th part each (D = 64: two at a time), their sums are added in
// order.  A part that saw nothing of the row has the weight 0, whatever lies in its place.
template <int D>
__global__ void __launch_bounds__(256) attn_tc_join_kernel(const __grid_constant__ TcArgs w) {
  constexpr int kQuads = D / 4, kLanes = 256 / kQuads;
  __shared__ float f_s[kAttnSms], warp_s[8];
  __shared__ float4 o_s[kLanes][kQuads], v_s[10][256];
  const AttnArgs &a = w.a;
  const int unit = blockIdx.x >> 8, r = blockIdx.x & 255, hv = unit % a.V, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = r & 127, rt = rr / a.G, tk = (r >> 7) * w.tokens + rt;
  pdl_release();
  pdl_wait();
  const int2 rows = __ldcg(w.rows + unit);
  if (rt >= w.tokens || tk >= rows.y) return;
  const int p = threadIdx.x;
  const float2 x = p < w.parts ? __ldcg(w.ml + ((size_t)unit * w.parts + p) * 256 + r) : make_float2(-INFINITY, 0.f);
  float mx = x.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) warp_s[warp] = mx;
  __syncthreads();
  mx = warp_s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, warp_s[i]);
  const float f = ex2(x.x - (mx == -INFINITY ? 0.f : mx));
  if (p < w.parts) f_s[p] = f;
  float sum = f * x.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if (lane == 0) warp_s[warp] = sum;
  const int q = threadIdx.x % kQuads, first = threadIdx.x / kQuads;
  const float4 *o = reinterpret_cast<const float4 *>(a.part + ((size_t)unit * w.parts * 256 + r) * D) + (q ^ (r & (kQuads - 1)));
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k0 = first; k0 < w.parts; k0 += 10 * kLanes) {
    // by way of shared memory: the compiler would wait for each load before it issues the next
#pragma unroll
    for (int i = 0; i < 10; ++i) cp_async16(&v_s[i][threadIdx.x], o + (size_t)min(k0 + i * kLanes, w.parts - 1) * 256 * kQuads);
    cp_async_wait_all();
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const int k = k0 + i * kLanes;
      const float g = k < w.parts ? f_s[k] : 0.f;
      const float4 v = g == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : v_s[i][threadIdx.x];
      y[0] += g * v.x;
      y[1] += g * v.y;
      y[2] += g * v.z;
      y[3] += g * v.w;
    }
  }
  o_s[first][q] = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (threadIdx.x >= kQuads) return;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) total += warp_s[i];
  float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const float4 v = o_s[i][q];
    z[0] += v.x;
    z[1] += v.y;
    z[2] += v.z;
    z[3] += v.w;
  }
  const float inv = total == 0.f ? 0.f : 1.0f / total;
  uint16_t *dst = a.out + ((size_t)(rows.x + tk) * a.H + (size_t)hv * a.G + rr - rt * a.G) * D + q * 4;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(z[0] * inv, z[1] * inv), pack_bf16x2(z[2] * inv, z[3] * inv));
}

// The same with a warp a row, for up to 32 parts, of which a lane has 10 in flight (D = 64: two half warps take turns).
// With 8 warps a row 16 items of 9 parts took 25 us, most of it waits of blocks that had one load each.
template <int D>
__global__ void __launch_bounds__(256) attn_tc_join_few_kernel(const __grid_constant__ TcArgs w) {
  constexpr int kQuads = D / 4, kLanes = 32 / kQuads;
  __shared__ float4 v_s[10][256];
  const AttnArgs &a = w.a;
  const int lane = threadIdx.x & 31, at = blockIdx.x * 8 + (threadIdx.x >> 5), unit = at >> 8, r = at & 255, hv = unit % a.V;
  const int rr = r & 127, rt = rr / a.G, tk = (r >> 7) * w.tokens + rt;
  pdl_release();
  pdl_wait();
  const int2 rows = __ldcg(w.rows + unit);
  const float2 x = lane < w.parts ? __ldcg(w.ml + ((size_t)unit * w.parts + lane) * 256 + r) : make_float2(-INFINITY, 0.f);
  if (rt >= w.tokens || tk >= rows.y) return;
  float mx = x.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float f = ex2(x.x - (mx == -INFINITY ? 0.f : mx));
  float sum = f * x.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int q = lane % kQuads, first = lane / kQuads;
  const float4 *o = reinterpret_cast<const float4 *>(a.part + ((size_t)unit * w.parts * 256 + r) * D) + (q ^ (r & (kQuads - 1)));
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k0 = 0; k0 < w.parts; k0 += 10 * kLanes) {
#pragma unroll
    for (int i = 0; i < 10; ++i)
      cp_async16(&v_s[i][threadIdx.x], o + (size_t)min(k0 + i * kLanes + first, w.parts - 1) * 256 * kQuads);
    cp_async_wait_all();
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const int k = k0 + i * kLanes + first;
      const float fk = __shfl_sync(0xffffffffu, f, k & 31), g = k < w.parts ? fk : 0.f;
      const float4 v = g == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : v_s[i][threadIdx.x];
      y[0] += g * v.x;
      y[1] += g * v.y;
      y[2] += g * v.z;
      y[3] += g * v.w;
    }
  }
  if constexpr (kLanes == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += __shfl_xor_sync(0xffffffffu, y[i], 16);
    if (first) return;
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  uint16_t *dst = a.out + ((size_t)(rows.x + tk) * a.H + (size_t)hv * a.G + rr - rt * a.G) * D + q * 4;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv));
}

template <int D>
cudaError_t launch_tc(const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s) {
  using C = TcCfg<D>;
  TcArgs w{a, kTcRows / a.G, 0, 0, nullptr, nullptr};
  auto fn = tma_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  CUtensorMap qm, km, vm;
  const cuuint32_t one[3] = {1, 1, 1};
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.ld_q * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)w.tokens};
    if (fn(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (!make_pages_map(&km, c.k, c.n_pages, a, D, kTcBK) || !make_pages_map(&vm, c.v, c.n_pages, a, D, kTcBK))
    return cudaErrorInvalidValue;
  const int pair = 2 * w.tokens;
  // m_1 + m_2 + ... = T of n sequences: the pairs of each, rounded up, are at most these
  const long long items = a.kv.q_start ? (a.T + (long long)std::min(a.T, a.kv.n_seqs) * (pair - 1)) / pair
                                       : (long long)a.kv.n_seqs * ((a.kv.per + pair - 1) / pair);
  if (items * a.V > 0x7fffffffll) return cudaErrorInvalidValue;
  // the key tiles of an item, at most
  const long long span = a.window > 0 ? std::min<long long>(a.kv.cap, (long long)a.window + pair + a.n_sinks) : a.kv.cap;
  const int tiles = (int)((span + kTcBK - 1) / kTcBK);
  // Clusters share the keys of an item where the items leave half of the SMs idle and the longest sequence gives every
  // CTA two key tiles.  Of 8 CTAs no more than 14 find room at once (16 items: two rounds, 86 us instead of 46).
  const int units = (int)(items * a.V);
  while (w.log_splits < 3 && (units << (w.log_splits + 1)) <= (w.log_splits == 2 ? 14 * 8 : kAttnSms) &&
         tiles >= 4 << w.log_splits)
    ++w.log_splits;
  // Parts without a cluster, joined by a second launch, may be any number: where that saves two steps of the longest
  // item (2 us each; the launch and its loads take about 4), or costs none and small clusters would share few items.
  // 16 tokens on 32768: 63 us with a cluster of 8, 18 so; 600 on 16000 141 and 104; 100 on 700 20.6 and 17.8; but 512
  // on 1500 21.4 and 24.3, 1024 alone 21 and 27.
  const int parts = units <= kAttnSms / 2 ? std::min(kAttnSms / units, tiles / 2) : 1;
  if (parts > 1) {
    const int with = (tiles + (1 << w.log_splits) - 1) >> w.log_splits, without = (tiles + parts - 1) / parts;
    if (without + 2 <= with || (without <= with && w.log_splits < 3 && units <= 12)) {
      w.parts = parts;
      w.log_splits = 0;
      w.ml = reinterpret_cast<float2 *>(a.part + (size_t)kAttnSms * 256 * D);
      w.rows = reinterpret_cast<int2 *>(w.ml + kAttnSms * 256);
    }
  }
  const unsigned splits = w.parts ? w.parts : 1u << w.log_splits;
  // the register shares have to be what the launch holds: raising them waits for what the others give up (and all
  // registers of an SM, so that no CTA of another launch holds tensor memory beside this one's)
  cudaFuncAttributes fa;
  cudaError_t err = cudaFuncGetAttributes(&fa, attn_tc_kernel<D>);
  if (err != cudaSuccess) return err;
  if (fa.numRegs * kTcThreads < 2 * 128 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)C::kSmemTiles * C::kTileBytes + sizeof(TcBars<D>) + 1024;
  err = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  err = launch_dependent(attn_tc_kernel<D>, (unsigned)(items * a.V) * splits, kTcThreads, smem, w.parts ? 1 : splits, s, qm,
                         km, vm, w);
  if (err != cudaSuccess || !w.parts) return err;
  if (w.parts <= 32) return launch_dependent(attn_tc_join_few_kernel<D>, (unsigned)units * 32, 256, 0, 1, s, w);
  return launch_dependent(attn_tc_join_kernel<D>, (unsigned)units * 256, 256, 0, 1, s, w);
}

}  // namespace

cudaError_t launch_attn_tc(const moe_attn_dims &d, const AttnArgs &a, const moe_kv_cache &c, cudaStream_t s) {
  return d.head_dim == 128 ? launch_tc<128>(a, c, s) : launch_tc<64>(a, c, s);
}

}  // namespace moe
