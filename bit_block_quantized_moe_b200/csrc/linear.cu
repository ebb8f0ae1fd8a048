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
// With an fp32 output K runs in slices of 256: each slice has a fresh accumulator, added in fp32 to a running sum in
// the epilogue's registers, because the tensor core's long accumulation truncates and loses up to 4e-6 of the result
// at K = 2048, which bf16 hides and fp32 does not.  When the tiles alone leave SMs idle, K is also split over CTAs
// and a second kernel adds the parts in split order.  Every wait is bounded (sync.cuh).
#include <algorithm>

#include "kernels.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kLnM = 128;         // features a tile
constexpr int kLnK = 64;          // K a chunk: one 128-byte swizzle row
constexpr int kLnSliceChunks = 4;  // chunks a slice, fp32 output
constexpr int kLnWave = 148;

template <int BN>
struct LnCfg {
  static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kCols = BN * 4 / kEpiWarps;  // columns an epilogue warp
  static constexpr int kABytes = kLnM * kLnK * 2;
  static constexpr int kBBytes = BN * kLnK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes > 8 ? 8 : 196608 / kStageBytes;
  static constexpr uint32_t kTmemCols = 2 * BN;
  static_assert(kStageBytes % 1024 == 0, "stages keep the 1024-byte alignment of the 128-byte swizzle");
};

template <int BN>
struct LnBars {
  uint64_t full[LnCfg<BN>::kStages], empty[LnCfg<BN>::kStages], dfull[2], dempty[2], done;
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
  float *part;  // [ks][T][N], ks > 1
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

__device__ __forceinline__ float ln_act(float z, int act) {
  if (act == MOE_ACT_SILU) return z / (1.0f + __expf(-z));
  if (act == MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}

__device__ __forceinline__ void ln_store(const LnArgs &a, size_t i, float z) {
  z = ln_act(z, a.act);
  if (a.resid)
    static_cast<float *>(a.out)[i] = a.resid[i] + z;
  else
    static_cast<uint16_t *>(a.out)[i] = float_to_bf16_bits(z);
}

template <int BN>
__global__ void __launch_bounds__(LnCfg<BN>::kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LnArgs a) {
  using C = LnCfg<BN>;
  extern __shared__ __align__(1024) uint8_t ln_raw[];
  uint8_t *smem = ln_raw + ((1024u - (smem_u32(ln_raw) & 1023u)) & 1023u);
  LnBars<BN> &B = *reinterpret_cast<LnBars<BN> *>(smem + C::kStages * C::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
  if (warp == 0) tmem_alloc(&B.tmem, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
      float run[C::kCols];
#pragma unroll
      for (int n = 0; n < C::kCols; ++n) run[n] = 0.f;
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
      const int f = ft * kLnM + 32 * q + lane;
      if (f < a.N) {
        const int t0 = tt * BN + part * C::kCols;
        if (a.ks > 1) {
          float *o = a.part + (size_t)ks * a.T * a.N;
#pragma unroll
          for (int n = 0; n < C::kCols; ++n)
            if (t0 + n < a.T) o[(size_t)(t0 + n) * a.N + f] = run[n];
        } else {
          const float b = a.bias ? a.bias[f] : 0.f;
#pragma unroll
          for (int n = 0; n < C::kCols; ++n)
            if (t0 + n < a.T) ln_store(a, (size_t)(t0 + n) * a.N + f, run[n] + b);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// The parts in split order, then the epilogue.
__global__ void linear_join_kernel(LnArgs a) {
  const size_t n = (size_t)a.T * a.N;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
    float z = a.part[i];
    for (int j = 1; j < a.ks; ++j) z += a.part[(size_t)j * n + i];
    ln_store(a, i, z + (a.bias ? a.bias[i % a.N] : 0.f));
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

template <int BN>
cudaError_t launch(const uint16_t *x, int64_t ld, const uint16_t *w, int K, LnArgs a, cudaStream_t s) {
  using C = LnCfg<BN>;
  CUtensorMap wmap, xmap;
  if (!make_matrix_map(&wmap, w, a.N, K, K, kLnM) || !make_matrix_map(&xmap, x, a.T, K, ld, BN))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)C::kStages * C::kStageBytes + sizeof(LnBars<BN>) + 1024;
  cudaError_t err = cudaFuncSetAttribute(linear_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  linear_kernel<BN><<<std::min(kLnWave, a.n_units), C::kThreads, smem, s>>>(wmap, xmap, a);
  return cudaGetLastError();
}

}  // namespace

size_t linear_part_bytes() { return (size_t)kLnWave * kLnM * 64 * 4; }

cudaError_t launch_linear(const uint16_t *x, int64_t ld, const uint16_t *w, const float *bias, int act,
                          const float *resid, void *out, int T, int K, int N, float *part, uint32_t *status,
                          cudaStream_t s) {
  LnArgs a{};
  a.T = T;
  a.N = N;
  a.n_ft = (N + kLnM - 1) / kLnM;
  a.chunks = (K + kLnK - 1) / kLnK;
  a.act = act;
  a.bias = bias;
  a.resid = resid;
  a.out = out;
  a.part = part;
  a.status = status;
  const int bn = T <= 16 ? 16 : (long long)a.n_ft * ((T + 127) / 128) < 74 ? 64 : 128;
  const int tiles = a.n_ft * ((T + bn - 1) / bn);
  a.ks = bn <= 64 ? std::max(1, std::min(kLnWave / tiles, (a.chunks + 3) / 4)) : 1;
  a.n_units = tiles * a.ks;
  a.slice = resid ? kLnSliceChunks : a.chunks;
  trace_mark(MOE_KERNEL_LINEAR, false, s);
  cudaError_t err = bn == 16   ? launch<16>(x, ld, w, K, a, s)
                    : bn == 64 ? launch<64>(x, ld, w, K, a, s)
                               : launch<128>(x, ld, w, K, a, s);
  if (err == cudaSuccess && a.ks > 1) {
    const size_t n = (size_t)T * N;
    linear_join_kernel<<<(unsigned)std::min<size_t>((n + 255) / 256, 1184), 256, 0, s>>>(a);
    err = cudaGetLastError();
  }
  trace_mark(MOE_KERNEL_LINEAR, true, s);
  return err;
}

}  // namespace moe
