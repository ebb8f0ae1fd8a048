// Matrix product with its epilogue on the 5th-generation tensor cores (tcgen05, sm_100a):
// out[t][f] = act(sum_k x[t][k] w[f][k] + bias[f]), bf16, or the fp32 residual plus that.
//
// A CTA tile is 128 features (tensor-memory lanes) x BN tokens (columns), so that an epilogue thread owns a feature
// (one bias register) and a warp writes 32 neighbouring features of a token at a time.
//   producer warp  : per 64-wide K chunk, TMA boxes of 128 weight rows and BN token rows (128-byte swizzle; rows
//                    past the end and columns past K read as zeros);
//   MMA warp       : 4 tcgen05.mma per chunk, both operands in shared memory; two accumulators in tensor memory, so
//                    that a tile's epilogue runs under the next tile's products;
//   epilogue warps : tensor memory lane quadrant = warp & 3; with 8 of them each has half of the columns.
// Many tiles of more than 128 features go to pairs of CTAs (tcgen05 cta_group::2): a pair's tile is 256 features x BN
// tokens, each CTA holds 128 weight rows, half of the token rows and the sums of its own features, and the first of
// them issues the products for both.  What a SM has to fetch through L2 per product, which bounds the single-CTA form
// (85 bytes a nanosecond a SM), falls by a third.
// With an fp32 output K runs in slices of 512: each slice has a fresh accumulator, added in fp32 to a running sum in
// the epilogue's registers, because the tensor core's long accumulation truncates: without a residual K = 2048 is
// 2.1e-6 of the result off and K = 4096 4.4e-6, which bf16 hides and fp32 does not; in slices of 512 it is 4.7e-7 at
// any K (an fp32 product in software: 3.9e-7 and 6.1e-7), in slices of 256 2.4e-7 but 14% slower.
// When the tiles alone leave SMs idle, a cluster of 2, 4 or 8 CTAs splits K: each sends the others their features'
// parts through distributed shared memory and finishes its own, summed in rank order.  Every wait on a barrier in shared
// memory is bounded (sync.cuh); CTAs of a cluster, which run together, meet without a limit.
// Measured: 32768 x 2048 x 2560 260 us in calls one behind another (1320 TFLOP/s at the clock that the power limit leaves;
// 231 us from idle, where single CTAs take 311); 1024 x 2048 x 2048 onto the residual 15.4 us, of which 7 are launch,
// first loads and epilogue; 3 x 2048 x 2560 5.7 us against 1.6 for reading the weights.
#include <algorithm>

#include "kernels.cuh"
#include "half.cuh"

namespace moe {
namespace {

constexpr int kLnM = 128;         // features a tile
constexpr int kLnK = 64;          // K a chunk: one 128-byte swizzle row
constexpr int kLnSliceChunks = 8;  // chunks a slice, fp32 output
constexpr int kLnWave = 148;

// SPLIT: clusters share K, a tile a CTA.  Otherwise persistent CTAs.
template <int BN, bool SPLIT>
struct LnCfg {
  static constexpr int kEpiWarps = BN >= 64 ? 8 : 4;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kCols = BN * 4 / kEpiWarps;  // columns an epilogue warp
  static constexpr int kABytes = kLnM * kLnK * 2;
  static constexpr int kBBytes = BN * kLnK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = SPLIT ? (BN == 64 ? 5 : 4) : BN == 256 ? 4 : 6;
  static constexpr int kSumBytes = SPLIT ? kLnM * BN * 4 : 0;  // the cluster's parts of this CTA's features
  static constexpr uint32_t kTmemCols = 2 * BN;
  static constexpr int kSumAt = kStages * kStageBytes;
  static constexpr int kBarsAt = kSumAt + kSumBytes;
  static_assert(kStageBytes % 1024 == 0, "stages keep the 1024-byte alignment of the 128-byte swizzle");
  static_assert(kBarsAt >= (BN == 16 ? 72 : BN == 64 ? 144 : 192) * 1024, "what may share an SM: see tmem_alloc below");
};

template <int STAGES>
struct LnBars {
  uint64_t full[STAGES], empty[STAGES], dfull[2], dempty[2], done;
  uint32_t tmem;
  int abort;
};

struct LnArgs {
  int T, N;
  int n_ft, n_units, ks, chunks;
  int slice;  // chunks a slice
  int act;
  const float *bias, *resid;
  void *out;
  uint32_t *status;
};

template <class Bars>
__device__ __forceinline__ bool ln_wait(uint64_t *bar, uint32_t parity, Bars &B, uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int *>(&B.abort)) return false;
  if (!mbar_wait(bar, parity)) {
    set_status(status, kStatusTimeout);
    B.abort = 1;
    return false;
  }
  return true;
}

// silu(z) = z / (1 + e^-z) with a power that cannot overflow, e = e^-|z|: z / (1 + e), and z e / (1 + e) below zero (the
// quotient by 1 + e^-z was cut to zero below -87, where the value is a normal number down to -91).
__device__ __forceinline__ float ln_silu(float z) {
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(fabsf(z) * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (z < 0.f ? z * e : z) * r;
}

// gelu(z) = z/2 (1 + erf(z / sqrt 2)) = (z + a)/2 - a F(-a), a = |z|, with the normal distribution F: 1 + erf would lose
// negative z (4% off at -5, nothing left at -5.6).  F(-a) = e^(-a^2/2) R(a), where R(a) = erfcx(a / sqrt 2)/2 falls from
// 1/2 as slowly as 1/a and is t P(t) with t = 1 / (1 + 0.3 a): a polynomial of degree 7, fitted by reweighted least
// squares to the smallest relative error (1.5e-7) over a <= 14, where F is below fp32's normal numbers.  Within
// (a^2 + 10) 2^-23 of the result.  32768 x 512 x 2560, which the epilogue bounds, takes 154 us; 179 with erff, and 249
// with erfcf, which does not cancel either.
__device__ __forceinline__ float ln_gelu(float z) {
  const float a = fminf(fabsf(z), 64.f);  // beyond, F is 0; infinities and NaN stay in the first term
  float t, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(a, 0.3f, 1.f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * a * -0.72134752f));  // -log2(e) / 2
  float p = 0.035674773f;
  p = fmaf(p, t, -0.15720308f);
  p = fmaf(p, t, 0.2063535f);
  p = fmaf(p, t, -0.053683642f);
  p = fmaf(p, t, 0.12856163f);
  p = fmaf(p, t, 0.09991349f);
  p = fmaf(p, t, 0.12075396f);
  p = fmaf(p, t, 0.1196293f);
  return fmaf(-(a * t), p * e, fmaf(0.5f, z, 0.5f * fabsf(z)));
}

// Finishes COUNT outputs i0, i0 + step, ... of sums z (with the bias in them), those with ok set: residuals are read
// together, before the first store, which may go to the same memory.
template <int COUNT>
__device__ __forceinline__ void ln_finish(const LnArgs &a, size_t i0, size_t step, float (&z)[COUNT], int ok) {
  if (a.act == MOE_ACT_SILU) {
#pragma unroll
    for (int n = 0; n < COUNT; ++n) z[n] = ln_silu(z[n]);
  } else if (a.act == MOE_ACT_GELU) {
#pragma unroll
    for (int n = 0; n < COUNT; ++n) z[n] = ln_gelu(z[n]);
  }
  if (a.resid) {
    float r[COUNT];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) r[n] = n < ok ? a.resid[i0 + n * step] : 0.f;
#pragma unroll
    for (int n = 0; n < COUNT; ++n)
      if (n < ok) static_cast<float *>(a.out)[i0 + n * step] = r[n] + z[n];
  } else {
#pragma unroll
    for (int n = 0; n < COUNT; ++n)
      if (n < ok) static_cast<uint16_t *>(a.out)[i0 + n * step] = float_to_bf16_bits(z[n]);
  }
}


// Sends COUNT tokens' sums of feature f of the tile, from token t0 of the tile on, to the rank that finishes the
// feature: [rank][token][feature of that rank].
template <int BN, int COUNT>
__device__ __forceinline__ void ln_send(uint8_t *sums, int ks, int f, int t0, const float (&z)[COUNT]) {
  const int own = kLnM / ks, to = f / own;
  const uint32_t at = cluster_map(smem_u32(sums), to) + (uint32_t)((cluster_rank() * BN + t0) * own + f - to * own) * 4u;
#pragma unroll
  for (int n = 0; n < COUNT; ++n) cluster_store(at + (uint32_t)(n * own) * 4u, z[n]);
}

// ---- pairs of CTAs ----
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *holder_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D[both CTAs' tensor memory] (+)= A[both CTAs' rows] * B[both CTAs' rows]^T, one K step of 16.
__device__ __forceinline__ void umma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs once the products issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A box to this CTA's memory, its bytes counted by the barrier at cluster address `bar` (the first CTA's).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int BN>
struct LnPairCfg {
  static constexpr int kThreads = 10 * 32;          // producer, products, 8 epilogue warps
  static constexpr int kCols = BN / 2;              // columns an epilogue warp
  static constexpr int kABytes = kLnM * kLnK * 2;
  static constexpr int kBBytes = BN / 2 * kLnK * 2; // this CTA's half of the token rows
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes;
  static constexpr int kBarsAt = kStages * kStageBytes;
};

template <int BN>
__global__ void __launch_bounds__(LnPairCfg<BN>::kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LnArgs a) {
  using C = LnPairCfg<BN>;
  extern __shared__ __align__(1024) uint8_t ln_raw[];
  // the same place in both CTAs: descriptors and barriers of one serve the other
  uint8_t *smem = ln_raw + ((1024u - (smem_u32(ln_raw) & 1023u)) & 1023u);
  LnBars<C::kStages> &B = *reinterpret_cast<LnBars<C::kStages> *>(smem + C::kBarsAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_release();
  const int rank = (int)cluster_rank(), first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.dfull[i], 1);
      mbar_init(&B.dempty[i], 16);  // both CTAs' epilogue warps (the first CTA's barrier)
    }
    mbar_init(&B.done, 1);
    B.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc_pair(&B.tmem, 2 * BN);
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // both CTAs' barriers are ready
  tc_fence_after();
  pdl_wait();
  const uint32_t tbase = B.tmem;

  if (warp == 0) {
    int cnt = 0, issued = 0;
    bool live = true;
    for (int u = first; u < a.n_units; u += step) {
      const int ft = u % a.n_ft, tt = u / a.n_ft;
      for (int c = 0; c < a.chunks; ++c, ++cnt) {
        const int s = cnt % C::kStages;
        if (live) live = __all_sync(0xffffffffu, ln_wait(&B.empty[s], ((cnt / C::kStages) & 1) ^ 1, B, a.status));
        if (!live) continue;
        issued = cnt + 1;
        if (elect_one()) {
          uint8_t *st = smem + s * C::kStageBytes;
          const uint32_t bar = cluster_map(smem_u32(&B.full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&B.full[s], 2u * C::kStageBytes);
          tma_load_2d_pair(st, &wmap, c * kLnK, ft * 256 + rank * kLnM, bar);
          tma_load_2d_pair(st + C::kABytes, &xmap, c * kLnK, tt * BN + rank * (BN / 2), bar);
        }
        __syncwarp();
      }
    }
    // Every copy issued must land before the CTAs exit: the first CTA's barriers count both CTAs' bytes.  (The second
    // CTA's copies are waited for by the first, and neither leaves before the other: the meeting at the end.)
    if (rank == 0)
      for (int c2 = max(0, issued - C::kStages); c2 < issued; ++c2)
        if (!mbar_wait(&B.full[c2 % C::kStages], (c2 / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = umma_idesc_bf16(256, BN);
      int cnt = 0, sc = 0;
      for (int u = first; u < a.n_units; u += step) {
        for (int c = 0; c < a.chunks;) {
          const int db = sc & 1;
          ln_wait(&B.dempty[db], ((sc >> 1) & 1) ^ 1, B, a.status);
          tc_fence_after();
          const uint32_t dcol = tbase + db * BN;
          const int e = min(a.chunks, c + a.slice);
          for (int c0 = c; c < e; ++c, ++cnt) {
            const int s = cnt % C::kStages;
            ln_wait(&B.full[s], (cnt / C::kStages) & 1, B, a.status);
            tc_fence_after();
            const uint32_t st = smem_u32(smem + s * C::kStageBytes);
            const uint64_t adesc = umma_sdesc_sw128(st), bdesc = umma_sdesc_sw128(st + C::kABytes);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < kLnK / 16; ++j)
                umma_ss_pair(dcol, adesc + 2 * j, bdesc + 2 * j, idesc, (c != c0) | (j != 0));
              umma_commit_pair(&B.empty[s]);
            }
            __syncwarp();
          }
          if (elect_one()) umma_commit_pair(&B.dfull[db]);
          __syncwarp();
          ++sc;
        }
      }
      // all products have completed before tensor memory is released
      if (elect_one()) {
        umma_commit_pair(&B.done);
        if (!mbar_wait(&B.done, 0)) set_status(a.status, kStatusTimeout);
      }
      __syncwarp();
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tcol = tbase + ((uint32_t)(32 * q) << 16) + part * C::kCols;
    const uint32_t dempty0 = cluster_map(smem_u32(&B.dempty[0]), 0), dempty1 = cluster_map(smem_u32(&B.dempty[1]), 0);
    int sc = 0;
    for (int u = first; u < a.n_units; u += step) {
      const int ft = u % a.n_ft, tt = u / a.n_ft;
      const int f = ft * 256 + rank * kLnM + 32 * q + lane, t0 = tt * BN + part * C::kCols;
      const float b = a.bias && f < a.N ? a.bias[f] : 0.f;
      if (BN == 256 || a.slice >= a.chunks) {
        ln_wait(&B.dfull[sc & 1], (sc >> 1) & 1, B, a.status);
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < C::kCols; h += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tcol + (sc & 1) * BN + h, v);
          tmem_wait_ld();
          float z[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) z[n] = __uint_as_float(v[n]) + b;
          if (f < a.N) ln_finish(a, (size_t)(t0 + h) * a.N + f, (size_t)a.N, z, a.T - t0 - h);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(sc & 1 ? dempty1 : dempty0);
        ++sc;
      } else if constexpr (BN == 128) {
        float run[C::kCols];
#pragma unroll
        for (int n = 0; n < C::kCols; ++n) run[n] = b;
        for (int c = 0; c < a.chunks; c += a.slice, ++sc) {
          ln_wait(&B.dfull[sc & 1], (sc >> 1) & 1, B, a.status);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < C::kCols; h += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tcol + (sc & 1) * BN + h, v);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < 32; ++n) run[h + n] += __uint_as_float(v[n]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(sc & 1 ? dempty1 : dempty0);
        }
#pragma unroll
        for (int h = 0; h < C::kCols; h += 32) {
          float z[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) z[n] = run[h + n];
          if (f < a.N) ln_finish(a, (size_t)(t0 + h) * a.N + f, (size_t)a.N, z, a.T - t0 - h);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (rank == 1 && warp == 1) mbar_wait(&B.done, 0);  // this CTA's copy of the last arrival (the first CTA reports)
  __syncwarp();
  cluster_meet();  // neither CTA leaves, or frees tensor memory, while the other's products or copies need it
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 2 * BN);
  }
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(LnCfg<BN, SPLIT>::kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LnArgs a) {
  using C = LnCfg<BN, SPLIT>;
  extern __shared__ __align__(1024) uint8_t ln_raw[];
  uint8_t *smem = ln_raw + ((1024u - (smem_u32(ln_raw) & 1023u)) & 1023u);
  LnBars<C::kStages> &B = *reinterpret_cast<LnBars<C::kStages> *>(smem + C::kBarsAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_release();

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.dfull[i], 1);
      mbar_init(&B.dempty[i], C::kEpiWarps);
    }
    mbar_init(&B.done, 1);
    B.abort = 0;
    mbar_fence_init();
  }
  // Tensor memory is taken before the wait (0.3 us earlier), although an earlier launch of the stream may have CTAs on
  // this SM that have yet to take theirs: shared memory lets at most tiles of 64 and 16, or 16 and 16, columns stand
  // together, 160 of 512 columns, and beside a CTA of attention's chunk kernel, which has all registers, nothing stands.
  if (warp == 0) tmem_alloc(&B.tmem, C::kTmemCols);
  tc_fence_before();
  if constexpr (SPLIT) cluster_meet();  // every CTA of the cluster is there before its memory is written
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tbase = B.tmem;

  if (warp == 0) {
    // The whole warp runs the loop on warp-uniform values; one elected lane issues the copies.
    int cnt = 0, issued = 0;
    bool live = true;
    for (int u = blockIdx.x; u < a.n_units; u += gridDim.x) {
      const int ks = u % a.ks, tile = u / a.ks, ft = tile % a.n_ft, tt = tile / a.n_ft;
      const int c1 = (int)((long long)a.chunks * (ks + 1) / a.ks);
      for (int c = (int)((long long)a.chunks * ks / a.ks); c < c1; ++c, ++cnt) {
        const int s = cnt % C::kStages;
        if (live) live = __all_sync(0xffffffffu, ln_wait(&B.empty[s], ((cnt / C::kStages) & 1) ^ 1, B, a.status));
        if (!live) continue;
        issued = cnt + 1;
        if (elect_one()) {
          uint8_t *st = smem + s * C::kStageBytes;
          mbar_arrive_expect_tx(&B.full[s], (uint32_t)C::kStageBytes);
          tma_load_2d(st, &wmap, c * kLnK, ft * kLnM, &B.full[s]);
          tma_load_2d(st + C::kABytes, &xmap, c * kLnK, tt * BN, &B.full[s]);
        }
        __syncwarp();
      }
    }
    // Every copy issued must land before the CTA exits, also after an abort (a bounded wait of its own).
    for (int c2 = max(0, issued - C::kStages); c2 < issued; ++c2)
      if (!mbar_wait(&B.full[c2 % C::kStages], (c2 / C::kStages) & 1)) set_status(a.status, kStatusTimeout);
  } else if (warp == 1) {
    const uint32_t idesc = umma_idesc_bf16(kLnM, BN);
    int cnt = 0, sc = 0;
    for (int u = blockIdx.x; u < a.n_units; u += gridDim.x) {
      const int ks = u % a.ks;
      const int c1 = (int)((long long)a.chunks * (ks + 1) / a.ks);
      int c = (int)((long long)a.chunks * ks / a.ks);
      while (c < c1) {
        const int db = sc & 1;
        ln_wait(&B.dempty[db], ((sc >> 1) & 1) ^ 1, B, a.status);
        tc_fence_after();
        const uint32_t dcol = tbase + db * BN;
        const int e = min(c1, c + a.slice);
        for (int first = c; c < e; ++c, ++cnt) {
          const int s = cnt % C::kStages;
          ln_wait(&B.full[s], (cnt / C::kStages) & 1, B, a.status);
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * C::kStageBytes);
          const uint64_t adesc = umma_sdesc_sw128(st), bdesc = umma_sdesc_sw128(st + C::kABytes);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < kLnK / 16; ++j)
              umma_ss(dcol, adesc + 2 * j, bdesc + 2 * j, idesc, (c != first) | (j != 0));
            umma_commit(&B.empty[s]);
          }
          __syncwarp();
        }
        if (elect_one()) umma_commit(&B.dfull[db]);
        __syncwarp();
        ++sc;
      }
    }
    // all MMAs issued by this warp have completed before tensor memory is released
    if (elect_one()) {
      umma_commit(&B.done);
      if (!mbar_wait(&B.done, 0)) set_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tcol = tbase + ((uint32_t)(32 * q) << 16) + part * C::kCols;
    constexpr int kStep = C::kCols < 32 ? C::kCols : 32;
    int sc = 0;
    for (int u = blockIdx.x; u < a.n_units; u += gridDim.x) {
      const int ks = u % a.ks, tile = u / a.ks, ft = tile % a.n_ft, tt = tile / a.n_ft;
      const int c1 = (int)((long long)a.chunks * (ks + 1) / a.ks);
      int c = (int)((long long)a.chunks * ks / a.ks);
      const int f = ft * kLnM + 32 * q + lane, t0 = tt * BN + part * C::kCols;
      const float b = a.bias && f < a.N ? a.bias[f] : 0.f;
      if (!SPLIT && BN == 256 || c + a.slice >= c1) {
        // one slice: straight out of tensor memory, a group of columns at a time
        ln_wait(&B.dfull[sc & 1], (sc >> 1) & 1, B, a.status);
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < C::kCols; h += kStep) {
          uint32_t v[32];
          if constexpr (kStep == 32)
            tmem_ld_32x32b_x32(tcol + (sc & 1) * BN + h, v);
          else
            tmem_ld_32x32b_x16(tcol + (sc & 1) * BN + h, v);
          tmem_wait_ld();
          float z[kStep];
#pragma unroll
          for (int n = 0; n < kStep; ++n) z[n] = __uint_as_float(v[n]);
          if constexpr (SPLIT) {
            ln_send<BN>(smem + C::kSumAt, a.ks, 32 * q + lane, part * C::kCols + h, z);
          } else {
#pragma unroll
            for (int n = 0; n < kStep; ++n) z[n] += b;
            if (f < a.N) ln_finish(a, (size_t)(t0 + h) * a.N + f, (size_t)a.N, z, a.T - t0 - h);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.dempty[sc & 1]);
        ++sc;
      } else if constexpr (BN <= 128) {
        float run[C::kCols];
#pragma unroll
        for (int n = 0; n < C::kCols; ++n) run[n] = SPLIT ? 0.f : b;
        for (; c < c1; c += a.slice, ++sc) {
          const int db = sc & 1;
          ln_wait(&B.dfull[db], (sc >> 1) & 1, B, a.status);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < C::kCols; h += kStep) {
            uint32_t v[32];
            if constexpr (kStep == 32)
              tmem_ld_32x32b_x32(tcol + db * BN + h, v);
            else
              tmem_ld_32x32b_x16(tcol + db * BN + h, v);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < kStep; ++n) run[h + n] += __uint_as_float(v[n]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.dempty[db]);
        }
#pragma unroll
        for (int h = 0; h < C::kCols; h += kStep) {
          float z[kStep];
#pragma unroll
          for (int n = 0; n < kStep; ++n) z[n] = run[h + n];
          if constexpr (SPLIT)
            ln_send<BN>(smem + C::kSumAt, a.ks, 32 * q + lane, part * C::kCols + h, z);
          else if (f < a.N)
            ln_finish(a, (size_t)(t0 + h) * a.N + f, (size_t)a.N, z, a.T - t0 - h);
        }
      }
    }
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_meet();  // the parts are there
    // this CTA's features, the ranks' parts in rank order
    const int tile = blockIdx.x / a.ks, ft = tile % a.n_ft, tt = tile / a.n_ft, own = kLnM / a.ks;
    const float *sums = reinterpret_cast<const float *>(smem + C::kSumAt);
    const int f0 = ft * kLnM + (int)cluster_rank() * own;
    for (int i = threadIdx.x; i < own * BN; i += C::kThreads) {
      const int f = f0 + i % own, t = tt * BN + i / own;
      if (f >= a.N || t >= a.T) continue;
      float z[1] = {a.bias ? a.bias[f] : 0.f};
      for (int r = 0; r < a.ks; ++r) z[0] += sums[r * own * BN + i];
      ln_finish(a, (size_t)t * a.N + f, 0, z, 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

bool make_matrix_map(CUtensorMap *map, const void *base, int rows, int cols, int64_t ld, int box_rows) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {kLnK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool SPLIT>
cudaError_t launch(const uint16_t *x, int64_t ld, const uint16_t *w, int K, const LnArgs &a, cudaStream_t s) {
  using C = LnCfg<BN, SPLIT>;
  CUtensorMap wmap, xmap;
  if (!make_matrix_map(&wmap, w, a.N, K, K, kLnM) || !make_matrix_map(&xmap, x, a.T, K, ld, BN))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)C::kBarsAt + sizeof(LnBars<C::kStages>) + 1024;
  cudaError_t err = cudaFuncSetAttribute(linear_kernel<BN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  return launch_dependent(linear_kernel<BN, SPLIT>, (unsigned)(SPLIT ? a.n_units : std::min(kLnWave, a.n_units)),
                          C::kThreads, smem, (unsigned)a.ks, s, wmap, xmap, a);
}

template <int BN>
cudaError_t launch_pair(const uint16_t *x, int64_t ld, const uint16_t *w, int K, LnArgs a, cudaStream_t s) {
  using C = LnPairCfg<BN>;
  CUtensorMap wmap, xmap;
  if (!make_matrix_map(&wmap, w, a.N, K, K, kLnM) || !make_matrix_map(&xmap, x, a.T, K, ld, BN / 2))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)C::kBarsAt + sizeof(LnBars<C::kStages>) + 1024;
  cudaError_t err = cudaFuncSetAttribute(linear_pair_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  return launch_dependent(linear_pair_kernel<BN>, 2u * std::min(kLnWave / 2, a.n_units), C::kThreads, smem, 2, s, wmap,
                          xmap, a);
}

}  // namespace

cudaError_t launch_linear(const uint16_t *x, int64_t ld, const uint16_t *w, const float *bias, int act,
                          const float *resid, void *out, int T, int K, int N, uint32_t *status, cudaStream_t s) {
  LnArgs a{};
  a.T = T;
  a.N = N;
  a.n_ft = (N + kLnM - 1) / kLnM;
  a.chunks = (K + kLnK - 1) / kLnK;
  a.act = act;
  a.bias = bias;
  a.resid = resid;
  a.out = out;
  a.status = status;
  // The tile that takes the fewest rounds of 64-wide chunks, each weighed by its products' cycles (64 columns are bound
  // by shared memory, 192 cycles); where the tiles leave half of the SMs idle, K split over a cluster (3 x 2048 x 2560:
  // 7.4 us with the parts through global memory and a second launch, 6.5 so).  Between the two, as 777 x 1160 x 1001 with
  // 104 tiles of 64 tokens, a CTA walks all of K alone.
  auto tiles = [&](int bn) { return (long long)a.n_ft * ((T + bn - 1) / bn); };
  int bn = 16;
  if (T > 16) {
    long long best = -1;
    for (int c : {64, 128, 256}) {
      if (c == 256 && resid) continue;
      const long long t = tiles(c), cost = (t + kLnWave - 1) / kLnWave * (c == 64 ? 192 : c);
      if (best < 0 || cost <= best) {
        best = cost;
        bn = c;
      }
    }
    if (bn == 256 && tiles(256) < kLnWave) bn = 128;
    if (bn == 128 && tiles(128) < kLnWave / 2) bn = 64;
  }
  a.ks = 1;
  a.slice = resid ? kLnSliceChunks : a.chunks;
  // Pairs of CTAs, once their tiles fill three quarters of the SMs.
  const int n_ft2 = (N + 255) / 256, pair = resid ? 128 : 256;
  for (int c = pair; c >= 128 && N > kLnM; c /= 2) {
    const long long t = (long long)n_ft2 * ((T + c - 1) / c);
    if (t * 4 < kLnWave / 2 * 3) continue;
    if (t > 0x7fffffffll) return cudaErrorInvalidValue;
    a.n_ft = n_ft2;
    a.n_units = (int)t;
    trace_mark(MOE_KERNEL_LINEAR, false, s);
    const cudaError_t err = c == 256 ? launch_pair<256>(x, ld, w, K, a, s) : launch_pair<128>(x, ld, w, K, a, s);
    trace_mark(MOE_KERNEL_LINEAR, true, s);
    return err;
  }
  while (bn <= 64 && a.ks < 8 && tiles(bn) * a.ks * 2 <= (bn == 16 ? 2 : 1) * kLnWave && a.chunks / (a.ks * 2) >= 2) a.ks *= 2;
  const long long units = tiles(bn) * a.ks;
  if (units > 0x7fffffffll) return cudaErrorInvalidValue;
  a.n_units = (int)units;
  trace_mark(MOE_KERNEL_LINEAR, false, s);
  cudaError_t err;
  if (a.ks > 1)
    err = bn == 16 ? launch<16, true>(x, ld, w, K, a, s) : launch<64, true>(x, ld, w, K, a, s);
  else
    err = bn == 16    ? launch<16, false>(x, ld, w, K, a, s)
          : bn == 64  ? launch<64, false>(x, ld, w, K, a, s)
          : bn == 128 ? launch<128, false>(x, ld, w, K, a, s)
                      : launch<256, false>(x, ld, w, K, a, s);
  trace_mark(MOE_KERNEL_LINEAR, true, s);
  return err;
}

}  // namespace moe
