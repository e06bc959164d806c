// int8 matrix product with one scale a token and one a channel:
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n],
// a [M, K] and w [N, K] int8 codes, K fastest; out bf16 or fp32.
//
// tcgen05.mma kind::i8 with int32 accumulators in TMEM: the sums are exact for
// K <= 32,768 (K 127^2 < 2^31), so neither the order of K nor a split of it
// changes a bit; the scales, the bias and one rounding follow in fp32.
//
// One CTA per SM walks over output tiles.  Warp 4 brings 128-byte K slices of
// both operands into a ring of shared-memory stages by TMA (128-byte swizzle;
// rows and bytes past an operand's end read as zero), warp 5 issues the MMAs,
// warps 0-3 turn a finished accumulator into output rows while the next tile
// accumulates into the other half of TMEM.
//
// The operand on the MMA's M side (128 rows, one TMEM lane each) is the tokens
// for many tokens, the weights for few (kSwap).
#include "bsa_device.cuh"
#include "bsa_kernels.h"

namespace bsa {

namespace {

constexpr int kThreads = 192;
constexpr int kSlice = 128;                 // bytes of K a stage
constexpr int kRowTile = 128;

template <int kCols>
struct LinearSmem {
  static constexpr int kRing = kCols >= 128 ? 6 : (kCols >= 64 ? 8 : 10);
  static constexpr uint32_t kA = kRowTile * kSlice, kB = kCols * kSlice;
  static constexpr uint32_t kCtl = kRing * (kA + kB);
  static constexpr uint32_t kBytes = kCtl + 256 + 1024;   // control, base alignment
};

struct LinearCtl {
  uint64_t full[10], empty[10], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(LinearCtl) <= 256, "control block");

// Tile order: columns of `kGroup` row tiles at a time, so that tiles in flight
// share operand rows in L2.
constexpr int kGroup = 16;
__device__ __forceinline__ void tile_of(int64_t t, int row_tiles, int col_tiles, int* r, int* c) {
  const int64_t per = static_cast<int64_t>(kGroup) * col_tiles;
  const int g = static_cast<int>(t / per);
  const int64_t in = t - g * per;
  const int rows = min(kGroup, row_tiles - g * kGroup);
  *r = g * kGroup + static_cast<int>(in % rows);
  *c = static_cast<int>(in / rows);
}

template <int kCols, bool kSwap>
__global__ void __launch_bounds__(kThreads, 1) linear_int8_kernel(
    const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_c,
    const LinearInt8Args a, int row_tiles, int col_tiles) {
  using S = LinearSmem<kCols>;
  constexpr int kRing = S::kRing;
  constexpr uint32_t kAccCols = kCols < 32 ? 32 : kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  LinearCtl* ctl = reinterpret_cast<LinearCtl*>(sm + S::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles = static_cast<int64_t>(row_tiles) * col_tiles;
  const int slices = (a.K + kSlice - 1) / kSlice;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], 128);
    }
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(&ctl->tmem_base, 2 * kAccCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx wc{&ctl->abort_flag, a.dev_status};

  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&map_r);
    prefetch_tensormap(&map_c);
    int64_t seq = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      int r, c;
      tile_of(t, row_tiles, col_tiles, &r, &c);
      for (int k = 0; k < slices; ++k, ++seq) {
        const int stage = static_cast<int>(seq % kRing);
        if (seq >= kRing && !mbar_wait(&ctl->empty[stage], ((seq / kRing) - 1) & 1, wc)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&ctl->full[stage], S::kA + S::kB);
        tma_load_2d(sm + stage * (S::kA + S::kB), &map_r, &ctl->full[stage], k * kSlice,
                    r * kRowTile);
        tma_load_2d(sm + stage * (S::kA + S::kB) + S::kA, &map_c, &ctl->full[stage], k * kSlice,
                    c * kCols);
      }
    }
    // every issued load has landed before the CTA exits
    for (int64_t k = (seq > kRing ? seq - kRing : 0); k < seq; ++k)
      mbar_wait(&ctl->full[k % kRing], (k / kRing) & 1, wc);
  } else if (warp == 5 && lane == 0) {
    const uint32_t id = idesc_s8_s32(kRowTile, kCols);
    int64_t seq = 0;
    int it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
      const int buf = it & 1;
      if (it >= 2 && !mbar_wait(&ctl->acc_empty[buf], ((it >> 1) - 1) & 1, wc)) break;
      tc_fence_after();
      for (int k = 0; k < slices; ++k, ++seq) {
        const int stage = static_cast<int>(seq % kRing);
        if (!mbar_wait(&ctl->full[stage], (seq / kRing) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ra = smem_u32(sm + stage * (S::kA + S::kB));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_s8_ss(tmem + buf * kAccCols, smem_desc_sw128(ra + kk * 32, 16, 1024),
                    smem_desc_sw128(ra + S::kA + kk * 32, 16, 1024), id, (k | kk) ? 1u : 0u);
        mma_commit(&ctl->empty[stage]);
      }
      if (ok) mma_commit(&ctl->acc_full[buf]);
    }
  } else if (warp < 4) {
    int it = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      const int buf = it & 1;
      int r, c;
      tile_of(t, row_tiles, col_tiles, &r, &c);
      if (!mbar_wait(&ctl->acc_full[buf], (it >> 1) & 1, wc)) break;
      tc_fence_after();
      const int row = r * kRowTile + warp * 32 + lane;   // a token, or a channel (kSwap)
      const uint32_t src = tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * kAccCols;
      const bool row_ok = row < (kSwap ? a.N : a.M);
      const float rs = row_ok ? __ldg((kSwap ? a.w_scale : a.a_scale) + row) : 0.f;
      const float rb = kSwap && row_ok && a.bias ? __ldg(a.bias + row) : 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 8) {
        uint32_t v[8];
        tmem_ld8(src + c0, v);
        tmem_wait_ld();
        const int col0 = c * kCols + c0;
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col0 + j;
          const bool in = col < (kSwap ? a.M : a.N);
          const float cs = in ? __ldg((kSwap ? a.a_scale : a.w_scale) + col) : 0.f;
          const float cb = !kSwap && in && a.bias ? __ldg(a.bias + col) : rb;
          // (sum * a_scale[m]) * w_scale[n] + bias, the same in both orders
          const float sum = static_cast<float>(static_cast<int32_t>(v[j]));
          o[j] = kSwap ? fmaf(sum * cs, rs, cb) : fmaf(sum * rs, cs, cb);
        }
        if (!row_ok) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col0 + j;
          if (col >= (kSwap ? a.M : a.N)) break;
          const int64_t at = kSwap ? col * a.ldo + row : row * a.ldo + col;
          if (a.out_fp32)
            static_cast<float*>(a.out)[at] = o[j];
          else
            static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o[j]);
        }
      }
      tc_fence_before();
      mbar_arrive(&ctl->acc_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, 2 * kAccCols);
}

template <int kCols, bool kSwap>
cudaError_t go(const LinearInt8Args& a, const CUtensorMap& mr, const CUtensorMap& mc,
               cudaStream_t st) {
  using S = LinearSmem<kCols>;
  auto* kernel = linear_int8_kernel<kCols, kSwap>;
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int rows = kSwap ? a.N : a.M, cols = kSwap ? a.M : a.N;
  const int rt = (rows + kRowTile - 1) / kRowTile, ct = (cols + kCols - 1) / kCols;
  const int64_t tiles = static_cast<int64_t>(rt) * ct;
  const int grid = tiles < 148 ? static_cast<int>(tiles) : 148;
  kernel<<<grid, kThreads, S::kBytes, st>>>(mr, mc, a, rt, ct);
  return cudaGetLastError();
}

}  // namespace

// Rows of the tensor maps' boxes (both 128 bytes wide): tokens and weights.
void linear_int8_boxes(int M, int* box_a, int* box_w) {
  *box_a = M <= 16 ? 16 : (M <= 64 ? 64 : 128);
  *box_w = 128;
}

cudaError_t launch_linear_int8(const LinearInt8Args& a, const CUtensorMap& ma,
                               const CUtensorMap& mw, cudaStream_t st) {
  if (a.M <= 16) return go<16, true>(a, mw, ma, st);
  if (a.M <= 64) return go<64, true>(a, mw, ma, st);
  return go<128, false>(a, ma, mw, st);
}

}  // namespace bsa
