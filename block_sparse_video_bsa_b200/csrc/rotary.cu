// Rotary positions of q, k and v rows, with the per-head RMS norm that comes
// before them and the change of layout to the attention's [B, H, N, 128].
//
// One row is a token's 128 dimensions of one head.  Pair i (of rotary_dim / 2)
// turns by theta = p_a(i) * f_i, p_a the token's position on the pair's axis:
//   (x0, x1) -> m (x0 cos - x1 sin, x1 cos + x0 sin),
// the other dimensions pass.  HBM-bound: every row is read once and written
// once, ten to twenty operations an element.  Measured: q, k and v of 37,740
// tokens and 56 heads, bf16, both norms: 506 us, 6.4 TB/s; 3 x 56 heads of 18,665
// tokens, 46 dimensions of the halves layout, no norm: 820 to 883 us, 5.5 to 5.9.
//
// Angles.  theta / 2 pi is kept as a 64-bit fixed-point fraction of a turn:
// step = f / (2 pi) mod 1 in units of 2^-64, computed once in fp64, and
// position * step wraps modulo 2^64 exactly as whole turns drop out.  Its top
// 32 bits go to sincospif.  So a position near 2^31 has the accuracy of a small
// one (fp64's 2^-53 on f, times the position, in turns), for one 64-bit
// multiply a pair instead of fp64 range reduction.
//
// A row is 8 lanes of two 8-dimension chunks.  In the halves layout with
// rotary_dim a multiple of 16 the lane's two chunks are each other's partners
// (i and i + rotary_dim / 16, in chunks), so both layouts turn inside a thread;
// only other rotary_dim of the halves layout exchange through shared memory.
// A CTA holds 32 rows at a time: `tt` consecutive tokens of 32 / tt heads, and
// walks over the heads of its chunk with the tokens fixed, so cos and sin (with
// the norm's weight folded in) are computed once for all of a chunk's heads and
// stay in registers.  Consecutive tokens of one head are written together: 8 KB
// runs of the head-major output.  Each thread keeps kDepth rows of its own on
// the way through shared memory with cp.async, so the bytes in flight do not
// cost registers, and no thread waits for another.
#include "bsa_device.cuh"
#include "bsa_kernels.h"

namespace bsa {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                  // threads a row
constexpr int kRows = kThreads / kLanes;   // rows a CTA holds at a time

enum { kInterleaved = 0, kHalfPaired = 1, kHalfAny = 2 };

// One lane's share of a row on its way: two chunks of 8 values.  Six bf16 or
// three fp32 rows a thread are 48 KB a CTA; less where the exchange takes room.
template <class T, int kMode>
struct Words {
  static constexpr int kPerChunk = sizeof(T) / 2;        // 16-byte words a chunk
  static constexpr int kDepth = (kMode == kHalfAny ? 4 : 6) / kPerChunk;
};

__device__ __forceinline__ void unpack8(const uint4* w, const __nv_bfloat16*, float x[8]) {
  bf16x8_to_f32(w[0], x);
}
__device__ __forceinline__ void unpack8(const uint4* w, const float*, float x[8]) {
  x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y);
  x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
  x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y);
  x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
}
// fp32 values, rounded once to the output type (to nearest even)
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float x[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void put8(float* p, const float x[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {   // a whole sector in one store
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The exchange buffer: a gap after every 8 values and rows of 152, so that a
// warp's four rows of eight lanes, 8 values apart, meet every bank once.
constexpr int kXchRow = 152;
__device__ __forceinline__ int xch_at(int e) { return e + (e >> 3); }

template <class Tin, int kMode>
constexpr int rotary_smem() {
  using W = Words<Tin, kMode>;
  return W::kDepth * 2 * W::kPerChunk * kThreads * 16 +
         (kMode == kHalfAny ? kRows * kXchRow * 4 : 0);
}

template <class Tin, class Tout, int kMode>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryArgs a) {
  constexpr int kW = Words<Tin, kMode>::kPerChunk, kDepth = Words<Tin, kMode>::kDepth;
  extern __shared__ uint4 dyn[];
  uint4 (*ring)[2 * kW][kThreads] = reinterpret_cast<uint4 (*)[2 * kW][kThreads]>(dyn);
  float (*xch)[kXchRow] = reinterpret_cast<float (*)[kXchRow]>(dyn + kDepth * 2 * kW * kThreads);
  const int lane = threadIdx.x & (kLanes - 1), row = threadIdx.x / kLanes;
  const int b = blockIdx.z / a.ntens, t = blockIdx.z % a.ntens;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * a.tt + (row & (a.tt - 1));
  const int hstep = kRows / a.tt;
  const int hb = blockIdx.y * a.hchunk;
  const int h_end = min(a.H, hb + a.hchunk);
  const int h0 = hb + row / a.tt;
  const int steps = (h_end - hb + hstep - 1) / hstep;   // the same for the whole CTA
  const bool live = n < a.N;
  const int r = a.r, half = r >> 1;
  const bool turns = a.turn[t] && r > 0;
  const bool norm = a.weight[t] != nullptr;

  // first dimensions of this lane's two chunks
  int e0 = lane * 8, e1 = lane * 8 + 64;
  if (kMode == kHalfPaired) {
    const int m = r >> 4;
    e0 = (lane < m ? lane : lane + m) * 8;        // the rest in order, so that 32-byte
    e1 = (lane < m ? lane + m : lane + 8) * 8;    // sectors are not split between the two
  }
  const Tin* src = static_cast<const Tin*>(a.in[t]) + b * a.in_b + n * a.in_n;
  Tout* dst = static_cast<Tout*>(a.out[t]) + b * a.out_b + n * a.out_n;

  auto fetch = [&](int j) {
    const int h = h0 + j * hstep;
    if (j < steps && live && h < h_end) {
      const Tin* p = src + h * a.in_h;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        cp_async16(&ring[j % kDepth][k][threadIdx.x], reinterpret_cast<const uint4*>(p + e0) + k, 16);
        cp_async16(&ring[j % kDepth][kW + k][threadIdx.x], reinterpret_cast<const uint4*>(p + e1) + k, 16);
      }
    }
    cp_async_commit();
  };
  grid_wait();
  grid_ready();
#pragma unroll
  for (int j = 0; j < kDepth - 1; ++j) fetch(j);

  // out = x c + partner s; sin carries the pair's sign, and the norm's weights
  // are folded in (s has the partner's)
  float c0[8], s0[8], c1[8], s1[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) c0[j] = c1[j] = 1.f, s0[j] = s1[j] = 0.f;
  // Steps of all pairs, once a CTA: fp64 runs at about one operation a clock and
  // SM, and a token of one head would need five for each of its pairs.  They lie
  // in the ring's last slot, which is filled only after the second barrier.
  uint64_t* steps64 = reinterpret_cast<uint64_t*>(&ring[kDepth - 1][0][0]);
  if (turns) {
    if (static_cast<int>(threadIdx.x) < half) {
      const double f = a.freqs[threadIdx.x] * 0.15915494309189533577;   // turns a position
      steps64[threadIdx.x] =
          static_cast<uint64_t>(__double2ll_rn((f - rint(f)) * 18446744073709551616.0));
    }
    __syncthreads();
  }
  if (turns && live) {
    const int32_t* pos = a.positions + b * a.pos_b + n * a.pos_n;
    auto turn = [&](int i, float* sn, float* cs) {
      int axis = 0;
      while (i >= a.axis_end[axis]) ++axis;
      const uint64_t phase =
          steps64[i] * static_cast<uint64_t>(static_cast<int64_t>(pos[axis]));
      // [-2^31, 2^31) of a turn in 2^-32 units -> half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, sn, cs);
      *cs *= a.scale;
      *sn *= a.sin_scale;
    };
    if (kMode == kInterleaved) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float sn, cs;
        if (e0 + j < r) {
          turn((e0 + j) >> 1, &sn, &cs);
          c0[j] = c0[j + 1] = cs, s0[j] = -sn, s0[j + 1] = sn;
        }
        if (e1 + j < r) {
          turn((e1 + j) >> 1, &sn, &cs);
          c1[j] = c1[j + 1] = cs, s1[j] = -sn, s1[j + 1] = sn;
        }
      }
    } else if (kMode == kHalfPaired) {
      if (e0 < half) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float sn, cs;
          turn(e0 + j, &sn, &cs);
          c0[j] = c1[j] = cs, s0[j] = -sn, s1[j] = sn;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float sn, cs;
        if (e0 + j < r) {
          turn(e0 + j < half ? e0 + j : e0 + j - half, &sn, &cs);
          c0[j] = cs, s0[j] = e0 + j < half ? -sn : sn;
        }
        if (e1 + j < r) {
          turn(e1 + j < half ? e1 + j : e1 + j - half, &sn, &cs);
          c1[j] = cs, s1[j] = e1 + j < half ? -sn : sn;
        }
      }
    }
  }
  if (turns) __syncthreads();
  if (norm) {
    const float* w = a.weight[t];
    auto partner = [&](int e) {
      if (kMode == kInterleaved) return e ^ 1;
      return e >= r ? e : (e < half ? e + half : e - half);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c0[j] *= w[e0 + j], s0[j] *= w[partner(e0 + j)];
      c1[j] *= w[e1 + j], s1[j] *= w[partner(e1 + j)];
    }
  }
  const bool part = r < kDim;   // some dimensions pass

  for (int j = 0; j < steps; ++j) {
    fetch(j + kDepth - 1);
    cp_async_wait<kDepth - 1>();
    const int h = h0 + j * hstep;
    const bool on = live && h < h_end;
    uint4 w[2 * kW];
#pragma unroll
    for (int k = 0; k < 2 * kW; ++k) w[k] = on ? ring[j % kDepth][k][threadIdx.x] : make_uint4(0, 0, 0, 0);
    Tout* p = dst + h * a.out_h;
    float x0[8], x1[8];
    unpack8(w, static_cast<const Tin*>(nullptr), x0);
    unpack8(w + kW, static_cast<const Tin*>(nullptr), x1);
    if (turns || norm) {
      float rs = 1.f;
      if (norm) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 u = make_float2(x0[i], x0[i + 1]), v = make_float2(x1[i], x1[i + 1]);
          q = fma2(v, v, fma2(u, u, q));
        }
        float ss = q.x + q.y;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * (1.f / kDim) + a.eps);
      }
      float y0[8], y1[8];
      if (kMode == kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y0[i] = x0[i ^ 1], y1[i] = x1[i ^ 1];
      } else if (kMode == kHalfPaired) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y0[i] = x1[i], y1[i] = x0[i];
      } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) xch[row][xch_at(e0 + i)] = x0[i], xch[row][xch_at(e1 + i)] = x1[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int u = e0 + i, v = e1 + i;
          y0[i] = xch[row][xch_at(u >= r ? u : (u < half ? u + half : u - half))];
          y1[i] = xch[row][xch_at(v >= r ? v : (v < half ? v + half : v - half))];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // dimensions past r pass (a 0 * infinity there would be NaN)
        const float u = x0[i] * c0[i], v = x1[i] * c1[i];
        const float tu = fmaf(y0[i], s0[i], u), tv = fmaf(y1[i], s1[i], v);
        x0[i] = part && e0 + i >= r ? u : tu;
        x1[i] = part && e1 + i >= r ? v : tv;
      }
      if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x0[i] *= rs, x1[i] *= rs;
      }
    }
    if (on) {
      put8(p + e0, x0);
      put8(p + e1, x1);
    }
  }
}

template <class Tin, class Tout, int kMode>
cudaError_t go(const RotaryArgs& a, dim3 grid, cudaStream_t st) {
  auto* kernel = rotary_kernel<Tin, Tout, kMode>;
  constexpr int bytes = rotary_smem<Tin, kMode>();
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  if (e != cudaSuccess) return e;
  return launch_early(kernel, grid, kThreads, bytes, st, 0, a);
}

template <class Tin, class Tout>
cudaError_t launch(const RotaryArgs& a, dim3 grid, cudaStream_t st) {
  if (a.interleaved) return go<Tin, Tout, kInterleaved>(a, grid, st);
  if (a.r % 16 == 0) return go<Tin, Tout, kHalfPaired>(a, grid, st);
  return go<Tin, Tout, kHalfAny>(a, grid, st);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, int in_fp32, int out_fp32, cudaStream_t st) {
  int tt = 1;
  while (tt < kRows && tt < a.N) tt *= 2;
  a.tt = tt;
  const int hstep = kRows / tt;
  const int64_t tiles = (static_cast<int64_t>(a.N) + tt - 1) / tt;
  // Split the heads until every SM has its CTAs; more would only repeat the
  // angles.
  const int64_t want = 148 * 3;
  int64_t chunks = (want + tiles * a.B * a.ntens - 1) / (tiles * a.B * a.ntens);
  const int most = (a.H + hstep - 1) / hstep;
  if (chunks > most) chunks = most;
  a.hchunk = (a.H + static_cast<int>(chunks) - 1) / static_cast<int>(chunks);
  a.hchunk = (a.hchunk + hstep - 1) / hstep * hstep;
  const dim3 grid(static_cast<unsigned>(tiles), (a.H + a.hchunk - 1) / a.hchunk, a.B * a.ntens);
  using bf16 = __nv_bfloat16;
  if (in_fp32) return out_fp32 ? launch<float, float>(a, grid, st) : launch<float, bf16>(a, grid, st);
  return out_fp32 ? launch<bf16, float>(a, grid, st) : launch<bf16, bf16>(a, grid, st);
}

}  // namespace bsa
