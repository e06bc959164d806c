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

// ------------------------------------------------------------ CTA pairs

// 256 tokens x kN channels a tile, computed by two CTAs as one MMA of 256 x kN
// x 32: each brings its 128 tokens and half of the channels, so an SM reads
// 128 + kN / 2 rows for 128 x kN products instead of 128 + kN.
constexpr int kPairThreads = 320;    // warps 0-7 epilogue, 8 producer, 9 MMA
constexpr int kPairRows = 256;

template <int kN>
struct PairSmem {
  static constexpr uint32_t kA = 128 * kSlice, kB = kN / 2 * kSlice;
  static constexpr int kRing = static_cast<int>((226 * 1024 - 1024 - 512) / (kA + kB));
  static constexpr uint32_t kCtl = kRing * (kA + kB);
  static constexpr uint32_t kBytes = kCtl + 512 + 1024;
};
struct PairCtl {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PairCtl) <= 512 && PairSmem<128>::kRing <= 12, "control block");

__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 output values of row `row`, columns col .. col + 31, from int32 sums.
__device__ __forceinline__ void finish32(const LinearInt8Args& a, int64_t row, int col, float rs,
                                         const uint32_t (&v)[32], bool wide) {
  if (wide && col + 32 <= a.N) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float o[16];
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 cs = __ldg(reinterpret_cast<const float4*>(a.w_scale + col + 16 * q + j));
        float4 cb = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.bias) cb = __ldg(reinterpret_cast<const float4*>(a.bias + col + 16 * q + j));
        const int at = 16 * q + j;
        const float2 p0 = mul2(make_float2(static_cast<int32_t>(v[at]), static_cast<int32_t>(v[at + 1])),
                               make_float2(rs, rs));
        const float2 p1 = mul2(make_float2(static_cast<int32_t>(v[at + 2]), static_cast<int32_t>(v[at + 3])),
                               make_float2(rs, rs));
        const float2 r0 = fma2(p0, make_float2(cs.x, cs.y), make_float2(cb.x, cb.y));
        const float2 r1 = fma2(p1, make_float2(cs.z, cs.w), make_float2(cb.z, cb.w));
        o[j] = r0.x, o[j + 1] = r0.y, o[j + 2] = r1.x, o[j + 3] = r1.y;
      }
      uint32_t w[8];
      if (a.out_fp32) {
        float* p = static_cast<float*>(a.out) + row * a.ldo + col + 16 * q;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(o[8 * h + j]);
          st_global_32(p + 8 * h, w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
        st_global_32(static_cast<__nv_bfloat16*>(a.out) + row * a.ldo + col + 16 * q, w);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (col + j < a.N) {
      const float cb = a.bias ? __ldg(a.bias + col + j) : 0.f;
      const float o = fmaf(static_cast<float>(static_cast<int32_t>(v[j])) * rs,
                           __ldg(a.w_scale + col + j), cb);
      if (a.out_fp32)
        static_cast<float*>(a.out)[row * a.ldo + col + j] = o;
      else
        static_cast<__nv_bfloat16*>(a.out)[row * a.ldo + col + j] = __float2bfloat16_rn(o);
    }
  }
}

template <int kN>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    linear_int8_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                            const __grid_constant__ CUtensorMap map_w, const LinearInt8Args a,
                            int row_tiles, int col_tiles, int wide) {
  using S = PairSmem<kN>;
  constexpr int kRing = S::kRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  PairCtl* ctl = reinterpret_cast<PairCtl*>(sm + S::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int64_t tiles = static_cast<int64_t>(row_tiles) * col_tiles;
  const int slices = (a.K + kSlice - 1) / kSlice;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ctl->full[i], 1);       // rank 0's counts the bytes of both CTAs
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], 16); // rank 0's: the epilogue warps of both
    }
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc_pair(&ctl->tmem_base, 2 * kN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx wc{&ctl->abort_flag, a.dev_status};

  if (warp == 8 && lane == 0) {
    // each CTA loads its own 128 rows of A and its half of the channels
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_w);
    uint32_t stage = 0, round = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      int r, c;
      tile_of(t, row_tiles, col_tiles, &r, &c);
      const int row = r * kPairRows + rank * 128, col = c * kN + rank * (kN / 2);
      for (int k = 0; k < slices; ++k) {
        if (round > 0 && !mbar_wait(&ctl->empty[stage], (round - 1) & 1, wc)) {
          ok = false;
          break;
        }
        if (rank == 0) mbar_arrive_expect_tx(&ctl->full[stage], 2 * (S::kA + S::kB));
        const uint32_t bar = map_to_rank(&ctl->full[stage], 0);
        uint8_t* dst = sm + stage * (S::kA + S::kB);
        tma_load_2d_pair(dst, &map_a, bar, k * kSlice, row);
        tma_load_2d_pair(dst + S::kA, &map_w, bar, k * kSlice, col);
        if (++stage == kRing) stage = 0, ++round;
      }
    }
  } else if (warp == 9 && lane == 0 && rank == 0) {
    const uint32_t id = idesc_s8_s32(kPairRows, kN);
    uint32_t stage = 0, round = 0;
    int it = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs, ++it) {
      const int buf = it & 1;
      if (it >= 2 && !mbar_wait(&ctl->acc_empty[buf], ((it >> 1) - 1) & 1, wc)) break;
      tc_fence_after();
      for (int k = 0; k < slices; ++k) {
        if (!mbar_wait(&ctl->full[stage], round & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ra = smem_u32(sm + stage * (S::kA + S::kB));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_s8_ss_pair(tmem + buf * kN, smem_desc_sw128(ra + kk * 32, 16, 1024),
                         smem_desc_sw128(ra + S::kA + kk * 32, 16, 1024), id, (k | kk) ? 1u : 0u);
        mma_commit_pair(&ctl->empty[stage]);
        if (++stage == kRing) stage = 0, ++round;
      }
      if (ok) mma_commit_pair(&ctl->acc_full[buf]);
    }
  } else if (warp < 8) {
    // warps w and w + 4 share TMEM lanes 32 (w % 4) .. + 31, a half of the columns each
    const int quad = warp & 3, side = warp >> 2;
    int it = 0;
    for (int64_t t = pair; t < tiles; t += pairs, ++it) {
      const int buf = it & 1;
      int r, c;
      tile_of(t, row_tiles, col_tiles, &r, &c);
      const int64_t row = static_cast<int64_t>(r) * kPairRows + rank * 128 + quad * 32 + lane;
      const bool row_ok = row < a.M;
      const float rs = row_ok ? __ldg(a.a_scale + row) : 0.f;
      if (!mbar_wait(&ctl->acc_full[buf], (it >> 1) & 1, wc)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kN;
#pragma unroll 1
      for (int c0 = side * (kN / 2); c0 < (side + 1) * (kN / 2); c0 += 32) {
        uint32_t v[32];
        BSA_TMEM_LD_32(src + c0, v);
        tmem_wait_ld();
        if (row_ok) finish32(a, row, c * kN + c0, rs, v, wide);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(&ctl->acc_empty[buf], 0));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no arrival of the peer is still on its way, nor its MMA reading here
  tc_fence_after();
  if (warp == 9) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 2 * kN);
  }
}

// Channels a tile: 256 unless 128 leave fewer SMs idle in the last wave.
int linear_pair_cols(int M, int N, int K) {
  auto waves = [&](int n) {
    const int64_t tiles = static_cast<int64_t>((M + kPairRows - 1) / kPairRows) * ((N + n - 1) / n);
    return (tiles + 73) / 74 * n;
  };
  return waves(256) <= waves(128) ? 256 : 128;
}

template <int kN>
cudaError_t go_pair(const LinearInt8Args& a, const CUtensorMap& ma, const CUtensorMap& mw,
                    cudaStream_t st) {
  using S = PairSmem<kN>;
  auto* kernel = linear_int8_pair_kernel<kN>;
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int rt = (a.M + kPairRows - 1) / kPairRows, ct = (a.N + kN - 1) / kN;
  const int64_t tiles = static_cast<int64_t>(rt) * ct;
  const int pairs = tiles < 74 ? static_cast<int>(tiles) : 74;
  const int size = a.out_fp32 ? 4 : 2;
  // 32-byte stores and 16-byte reads of the channels' scales and biases
  const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.ldo * size % 32 == 0 &&
                    reinterpret_cast<uintptr_t>(a.w_scale) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  kernel<<<2 * pairs, kPairThreads, S::kBytes, st>>>(ma, mw, a, rt, ct, wide);
  return cudaGetLastError();
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
void linear_int8_boxes(int M, int N, int K, int* box_a, int* box_w) {
  *box_a = M <= 16 ? 16 : (M <= 64 ? 64 : 128);
  *box_w = M <= 64 ? 128 : (linear_pair_cols(M, N, K) / 2);
}

cudaError_t launch_linear_int8(const LinearInt8Args& a, const CUtensorMap& ma,
                               const CUtensorMap& mw, cudaStream_t st) {
  if (a.M <= 16) return go<16, true>(a, mw, ma, st);
  if (a.M <= 64) return go<64, true>(a, mw, ma, st);
  return linear_pair_cols(a.M, a.N, a.K) == 256 ? go_pair<256>(a, ma, mw, st)
                                                : go_pair<128>(a, ma, mw, st);
}

}  // namespace bsa
