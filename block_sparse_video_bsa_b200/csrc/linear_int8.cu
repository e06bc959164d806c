// int8 matrix product with one scale a token and one a channel:
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n],
// a [M, K] and w [N, K] int8 codes, K fastest; out bf16 or fp32.
//
// tcgen05.mma kind::i8 with int32 accumulators in TMEM: the sums are exact for
// K <= 32,768 (K 127^2 < 2^31), so neither the order of K nor a split of it
// changes a bit; the scales, the bias and one rounding follow in fp32.
//
// Two kernels, both with TMA for the operands (128-byte K slices, 128-byte
// swizzle; rows and bytes past an operand's end read as zero), a ring of
// shared-memory stages, one thread that issues the MMAs and warps that turn
// accumulators into output:
//   linear_int8_pair_kernel  many tokens: CTA pairs, tokens on the MMA's M side;
//   linear_int8_few_kernel   up to 64 tokens: the weights on the M side, K split
//                            over a cluster.
#include "bsa_device.cuh"
#include "bsa_kernels.h"

namespace bsa {

namespace {

constexpr int kSlice = 128;                 // bytes of K a stage
constexpr int kRowTile = 128;

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

// ------------------------------------------------------------ few tokens

// 128 channels x kCols tokens a tile, the weights on the MMA's M side.  What
// bounds it is the stream of weights, so a cluster of CTAs splits K: each sums
// its share of the slices, keeps the int32 partial sums in shared memory, and
// the cluster adds them over distributed shared memory (whole numbers: the
// order does not matter).  No workspace, no atomics.
constexpr int kFewThreads = 192;     // warps 0-3 epilogue, 4 producer, 5 MMA
constexpr int kMaxSplit = 8;

template <int kCols>
struct FewSmem {
  static constexpr uint32_t kA = kRowTile * kSlice, kB = kCols * kSlice;
  static constexpr uint32_t kSums = kCols * kRowTile * 4;
  // two CTAs an SM
  static constexpr uint32_t kRoom = 111 * 1024 - 512 - 1024 - kSums;
  static constexpr int kRing = static_cast<int>(kRoom / (kA + kB));
  static constexpr uint32_t kOffSums = kRing * (kA + kB);
  static constexpr uint32_t kCtl = kOffSums + kSums;
  static constexpr uint32_t kBytes = kCtl + 512 + 1024;   // control, base alignment
};
struct FewCtl {
  uint64_t full[8], empty[8], acc_full, fin;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(FewCtl) <= 512 && FewSmem<16>::kRing <= 8 && FewSmem<64>::kRing <= 8,
              "control block");

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int kCols>
__global__ void __launch_bounds__(kFewThreads, 1) linear_int8_few_kernel(
    const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
    const LinearInt8Args a, int split) {
  using S = FewSmem<kCols>;
  constexpr int kRing = S::kRing;
  constexpr uint32_t kAccCols = kCols < 32 ? 32 : kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  FewCtl* ctl = reinterpret_cast<FewCtl*>(sm + S::kCtl);
  int32_t* sums = reinterpret_cast<int32_t*>(sm + S::kOffSums);   // [kCols][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x / split, rank = blockIdx.x % split;    // one cluster a row tile
  const int slices = (a.K + kSlice - 1) / kSlice;
  const int k0 = static_cast<int>(static_cast<int64_t>(slices) * rank / split);
  const int k1 = static_cast<int>(static_cast<int64_t>(slices) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->fin, 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(&ctl->tmem_base, kAccCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait();
  grid_ready();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx wc{&ctl->abort_flag, a.dev_status};

  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_a);
    uint32_t stage = 0, round = 0;
    for (int k = k0; k < k1; ++k) {
      if (round > 0 && !mbar_wait(&ctl->empty[stage], (round - 1) & 1, wc)) break;
      mbar_arrive_expect_tx(&ctl->full[stage], S::kA + S::kB);
      uint8_t* dst = sm + stage * (S::kA + S::kB);
      tma_load_2d(dst, &map_w, &ctl->full[stage], k * kSlice, r * kRowTile);
      tma_load_2d(dst + S::kA, &map_a, &ctl->full[stage], k * kSlice, 0);
      if (++stage == kRing) stage = 0, ++round;
    }
    // every issued load has landed before the CTA exits
    const int issued = static_cast<int>(round) * kRing + static_cast<int>(stage);
    for (int k = (issued > kRing ? issued - kRing : 0); k < issued; ++k)
      mbar_wait(&ctl->full[k % kRing], (k / kRing) & 1, wc);
  } else if (warp == 5 && lane == 0) {
    const uint32_t id = idesc_s8_s32(kRowTile, kCols);
    uint32_t stage = 0, round = 0;
    bool ok = true;
    for (int k = k0; k < k1; ++k) {
      if (!mbar_wait(&ctl->full[stage], round & 1, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t ra = smem_u32(sm + stage * (S::kA + S::kB));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_s8_ss(tmem, smem_desc_sw128(ra + kk * 32, 16, 1024),
                  smem_desc_sw128(ra + S::kA + kk * 32, 16, 1024), id, (k > k0 || kk) ? 1u : 0u);
      mma_commit(&ctl->empty[stage]);
      if (++stage == kRing) stage = 0, ++round;
    }
    if (ok) {
      mma_commit(&ctl->acc_full);
    } else {   // those that were issued end before TMEM is freed
      mma_commit(&ctl->fin);
      mbar_wait(&ctl->fin, 0, wc);
    }
  } else if (warp < 4) {
    // this share's sums, [token][channel]
    if (mbar_wait_warp(&ctl->acc_full, 0, wc)) {
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 8) {
        uint32_t v[8];
        tmem_ld8(src + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sums[(c0 + j) * kRowTile + warp * 32 + lane] = static_cast<int32_t>(v[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();
  // sums of a CTA whose waits ran out are none: its cluster leaves the tile unwritten
  const int ran_out = lane < split ? ld_cluster_s32(map_to_rank(&ctl->abort_flag, lane)) : 0;
  if (warp < 4 && __all_sync(0xffffffffu, ran_out == 0)) {
    // warp w of rank q finishes tokens q + split (w + 4 i), four neighbouring channels a lane
    const int ch = r * kRowTile + 4 * lane;
    float ws[4], cb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ws[j] = ch + j < a.N ? a.w_scale[ch + j] : 0.f;
      cb[j] = ch + j < a.N && a.bias ? a.bias[ch + j] : 0.f;
    }
    for (int m = rank + split * warp; m < kCols && m < a.M; m += 4 * split) {
      int4 sum = make_int4(0, 0, 0, 0);
      const int32_t* at = sums + m * kRowTile + 4 * lane;
      if (split == 1) {
        sum = *reinterpret_cast<const int4*>(at);
      } else {
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q) {
          if (q < split) {
            const int4 p = ld_cluster_v4(map_to_rank(at, q));
            sum.x += p.x, sum.y += p.y, sum.z += p.z, sum.w += p.w;
          }
        }
      }
      const float rs = a.a_scale[m];
      const float o[4] = {fmaf(static_cast<float>(sum.x) * rs, ws[0], cb[0]),
                          fmaf(static_cast<float>(sum.y) * rs, ws[1], cb[1]),
                          fmaf(static_cast<float>(sum.z) * rs, ws[2], cb[2]),
                          fmaf(static_cast<float>(sum.w) * rs, ws[3], cb[3])};
      const int64_t to = m * a.ldo + ch;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (ch + j < a.N) {
          if (a.out_fp32)
            static_cast<float*>(a.out)[to + j] = o[j];
          else
            static_cast<__nv_bfloat16*>(a.out)[to + j] = __float2bfloat16_rn(o[j]);
        }
      }
    }
  }
  if (split > 1) cluster_sync();   // the peers have read this CTA's sums
  if (warp == 5) {
    __syncwarp();
    tmem_dealloc(tmem, kAccCols);
  }
}

// CTAs a cluster: as many as keep all clusters on the GPU at once with room to
// place them, 224 CTAs (1 x 7,168 x 7,168, 56 row tiles: 18.3 us unsplit, 14.4
// in 2, 13.7 in 3 or 4, 15.1 in 5, 18 in 6; 168 row tiles: 29.0 us unsplit,
// 34.9 in 2).
int few_split(int row_tiles, int slices) {
  int s = row_tiles < 224 ? 224 / row_tiles : 1;
  if (s > kMaxSplit) s = kMaxSplit;
  return s < slices ? s : slices;
}

template <int kCols>
cudaError_t go_few(const LinearInt8Args& a, const CUtensorMap& mw, const CUtensorMap& ma,
                   cudaStream_t st) {
  using S = FewSmem<kCols>;
  auto* kernel = linear_int8_few_kernel<kCols>;
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int rt = (a.N + kRowTile - 1) / kRowTile;
  const int split = few_split(rt, (a.K + kSlice - 1) / kSlice);
  return launch_early(kernel, dim3(split * rt), kFewThreads, S::kBytes, st, split, mw, ma, a, split);
}

// ------------------------------------------------------------ CTA pairs

// 256 tokens x kN channels a tile, computed by two CTAs as one MMA of 256 x kN
// x 32: each brings its 128 tokens and half of the channels, so an SM reads
// 128 + kN / 2 rows for 128 x kN products instead of 128 + kN (one CTA of 128 x
// 128 took 3,650 us for 37,740 x 7,168 x 7,168, where shared-memory bandwidth
// bounds it; pairs of 256 x 256 take 1,190 to 1,430 us, 2.7 to 3.3 POP/s with
// the clock under the power cap).  Persistent: warp 8 loads, warp 9 of CTA 0
// issues, warps 0-7 finish a tile while the next accumulates into the other
// half of TMEM.
constexpr int kPairThreads = 320;    // warps 0-7 epilogue, 8 producer, 9 MMA
constexpr int kPairRows = 256;
constexpr int kTable = 128;          // columns of an epilogue warp

template <int kN>
struct PairSmem {
  static constexpr uint32_t kA = 128 * kSlice, kB = kN / 2 * kSlice;
  static constexpr uint32_t kStaging = 8 * 32 * 33 * 4;     // a 32 x 32 block, or the table, a warp
  static constexpr int kRing = static_cast<int>((227 * 1024 - 1024 - 512 - kStaging) / (kA + kB));
  static constexpr uint32_t kOffStaging = kRing * (kA + kB);
  static constexpr uint32_t kCtl = kOffStaging + kStaging;
  static constexpr uint32_t kBytes = kCtl + 512 + 1024;
};
struct PairCtl {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2], fin;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PairCtl) <= 512 && PairSmem<128>::kRing <= 12, "control block");

__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 output values of row `row`, columns col .. col + 31, from int32 sums: one
// row a thread, whole 32-byte sectors.
// scales, biases: of these columns, in shared memory.
__device__ __forceinline__ void finish_row(const LinearInt8Args& a, int64_t row, int col, float rs,
                                           const uint32_t (&v)[32], const float* scales,
                                           const float* biases) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float o[16];
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 cs = *reinterpret_cast<const float4*>(scales + 16 * q + j);
      const float4 cb = *reinterpret_cast<const float4*>(biases + 16 * q + j);
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
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A warp's block of 32 rows (lane: row row0 + lane, its 32 sums in v) and
// columns col .. col + 31 where rows start anywhere or the block is cut off:
// through shared memory, so that a row is written by neighbouring lanes.
__device__ __forceinline__ void finish_block(const LinearInt8Args& a, int64_t row0, int col,
                                             float rs, const uint32_t (&v)[32], float* stage) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = static_cast<float>(static_cast<int32_t>(v[j])) * rs;
  __syncwarp();
  const bool in = col + lane < a.N;
  const float cs = in ? a.w_scale[col + lane] : 0.f;
  const float cb = in && a.bias ? a.bias[col + lane] : 0.f;
  const int64_t at = row0 * a.ldo + col + lane;
  const int rows = in ? static_cast<int>(a.M - row0 < 32 ? a.M - row0 : 32) : 0;
  auto put = [&](auto* p) {
#pragma unroll 16
    for (int i = 0; i < rows; ++i, p += a.ldo) store_out(p, fmaf(stage[i * 33 + lane], cs, cb));
  };
  if (a.out_fp32)
    put(static_cast<float*>(a.out) + at);
  else
    put(static_cast<__nv_bfloat16*>(a.out) + at);
  __syncwarp();
}

template <int kN>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    linear_int8_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                            const __grid_constant__ CUtensorMap map_w, const LinearInt8Args a,
                            int row_tiles, int col_tiles, int wide) {
  using S = PairSmem<kN>;
  constexpr int kRing = S::kRing;
  constexpr int kBuf = kN > 128 ? 256 : 128;      // TMEM columns of a tile's sums
  constexpr int kSide = (kN / 32 + 1) / 2 * 32;   // columns of warps 0-3; the rest are warps 4-7's
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
    mbar_init(&ctl->fin, 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc_pair(&ctl->tmem_base, kN > 128 ? 512 : 256);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  grid_wait();
  grid_ready();
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
    // every issued load has landed before the CTAs exit (rank 0's barriers count both)
    if (rank == 0) {
      const int64_t issued = static_cast<int64_t>(round) * kRing + stage;
      for (int64_t k = issued > kRing ? issued - kRing : 0; k < issued; ++k)
        mbar_wait(&ctl->full[k % kRing], static_cast<uint32_t>(k / kRing) & 1, wc);
    }
  } else if (warp == 9 && lane == 0 && rank == 0) {
    const uint32_t id = idesc_s8_s32(kPairRows, kN);
    uint32_t stage = 0, round = 0;
    int it = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs, ++it) {
      const int buf = it & 1;
      if (it >= 2 && !mbar_wait(&ctl->acc_empty[buf], ((it >> 1) - 1) & 1, wc)) {
        ok = false;
        break;
      }
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
          mma_s8_ss_pair(tmem + buf * kBuf, smem_desc_sw128(ra + kk * 32, 16, 1024),
                         smem_desc_sw128(ra + S::kA + kk * 32, 16, 1024), id, (k | kk) ? 1u : 0u);
        mma_commit_pair(&ctl->empty[stage]);
        if (++stage == kRing) stage = 0, ++round;
      }
      if (ok) mma_commit_pair(&ctl->acc_full[buf]);
    }
    if (!ok) {   // those that were issued end before TMEM is freed
      mma_commit_pair(&ctl->fin);
      mbar_wait(&ctl->fin, 0, wc);
    }
  } else if (warp < 8) {
    // warps w and w + 4 share TMEM lanes 32 (w % 4) .. + 31, some of the columns each
    const int quad = warp & 3, side = warp >> 2;
    float* stage = reinterpret_cast<float*>(sm + S::kOffStaging) + warp * 32 * 33;
    int it = 0;
    for (int64_t t = pair; t < tiles; t += pairs, ++it) {
      const int buf = it & 1;
      int r, c;
      tile_of(t, row_tiles, col_tiles, &r, &c);
      const int64_t row = static_cast<int64_t>(r) * kPairRows + rank * 128 + quad * 32 + lane;
      const bool row_ok = row < a.M;
      const float rs = row_ok ? a.a_scale[row] : 0.f;
      if (wide) {
        // this warp's columns' scales and biases, on their way while the tile accumulates
        float* tab = stage;
        const int col = c * kN + side * kSide + 4 * lane;
        if (4 * lane < kSide) {
          float4 cs = make_float4(0.f, 0.f, 0.f, 0.f), cb = cs;
          if (col + 4 <= a.N) {
            cs = *reinterpret_cast<const float4*>(a.w_scale + col);
            if (a.bias) cb = *reinterpret_cast<const float4*>(a.bias + col);
          }
          reinterpret_cast<float4*>(tab)[lane] = cs;
          reinterpret_cast<float4*>(tab + kTable)[lane] = cb;
        }
        __syncwarp();
      }
      if (!mbar_wait_warp(&ctl->acc_full[buf], (it >> 1) & 1, wc)) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kBuf;
#pragma unroll 1
      for (int c0 = side * kSide; c0 < (side ? kN : kSide); c0 += 32) {
        uint32_t v[32];
        BSA_TMEM_LD_32(src + c0, v);
        tmem_wait_ld();
        const int col = c * kN + c0;
        if (wide && col + 32 <= a.N) {
          const float* tab = stage + c0 - side * kSide;
          if (row_ok) finish_row(a, row, col, rs, v, tab, tab + kTable);
          __syncwarp();
        } else if (col < a.N) {
          // a cut block behind whole ones: the table has served
          __syncwarp();
          finish_block(a, row - lane, col, rs, v, stage);
        }
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
    tmem_dealloc_pair(tmem, kN > 128 ? 512 : 256);
  }
}

// Channels a tile: those whose waves of 74 pairs cost least, a tile's cost going
// with the rows that an SM reads for it, 128 + channels / 2 (measured within a
// tenth over 16 shapes).  256 for many tiles (37,740 x 7,168 x 7,168: 1,233 us
// against 1,294 with 224); fewer where that fills the last wave (512 x 7,168 x
// 21,504: 57.7 with 224 and 60.0; 512 x 7,168 x 7,168: 21.2 and 23.9; 128 x
// 7,168 x 21,504: 34.3 with 160 and 42.9; 256 x 7,168 x 7,168: 18.7 with 128 and
// 21.6).
int linear_pair_cols(int M, int N) {
  const int64_t rows = (M + kPairRows - 1) / kPairRows;
  int best = 256;
  int64_t least = INT64_MAX;
  for (int cols = 256; cols >= 128; cols -= 32) {
    const int64_t waves = (rows * ((N + cols - 1) / cols) + 73) / 74;
    const int64_t cost = waves * (128 + cols / 2);
    if (cost < least) best = cols, least = cost;
  }
  return best;
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
  return launch_early(kernel, dim3(2 * pairs), kPairThreads, S::kBytes, st, 0, ma, mw, a, rt, ct,
                      static_cast<int>(wide));
}

}  // namespace

// Few tokens: 64 x 7,168 x 7,168 take 17.8 us with the channels on the M side and 20.6 us as a pair's
// tile; 128 take 30.8 and 21.2.
constexpr int kFewTokens = 64;

// Rows of the tensor maps' boxes (both 128 bytes wide): tokens and weights.
void linear_int8_boxes(int M, int N, int* box_a, int* box_w) {
  *box_a = M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128));
  *box_w = M <= kFewTokens ? 128 : linear_pair_cols(M, N) / 2;
}

cudaError_t launch_linear_int8(const LinearInt8Args& a, const CUtensorMap& ma,
                               const CUtensorMap& mw, cudaStream_t st) {
  if (a.M <= 16) return go_few<16>(a, mw, ma, st);
  if (a.M <= 32) return go_few<32>(a, mw, ma, st);
  if (a.M <= kFewTokens) return go_few<64>(a, mw, ma, st);
  switch (linear_pair_cols(a.M, a.N)) {
    case 128: return go_pair<128>(a, ma, mw, st);
    case 160: return go_pair<160>(a, ma, mw, st);
    case 192: return go_pair<192>(a, ma, mw, st);
    case 224: return go_pair<224>(a, ma, mw, st);
    default: return go_pair<256>(a, ma, mw, st);
  }
}

}  // namespace bsa
