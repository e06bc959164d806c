// Rotary positions of q, k and v rows, with the per-head RMS norm that comes
// before them and the change of layout to the attention's [B, H, N, 128].
//
// One row is a token's 128 dimensions of one head.  Pair i (of rotary_dim / 2)
// turns by theta = p_a(i) * f_i, p_a the token's position on the pair's axis:
//   (x0, x1) -> m (x0 cos - x1 sin, x1 cos + x0 sin),
// the other dimensions pass.  HBM-bound: every row is read once and written
// once, a few dozen operations an element.
//
// Angles.  theta / 2 pi is kept as a 64-bit fixed-point fraction of a turn:
// step = f / (2 pi) mod 1 in units of 2^-64, computed once in fp64, and
// position * step wraps modulo 2^64 exactly as whole turns drop out.  Its top
// 32 bits go to sincospif.  So a position near 2^31 has the accuracy of a small
// one (fp64's 2^-53 on f, times the position, in turns), for one 64-bit
// multiply a pair instead of fp64 range reduction.
//
// A row is 16 lanes of 8 dimensions (16-byte loads and stores for bf16).  A CTA
// holds 16 rows at a time: `tt` consecutive tokens of 16 / tt heads, and walks
// over the heads of its chunk with the tokens fixed, so cos and sin are
// computed once for all of a chunk's heads and stay in registers.  Consecutive
// tokens of one head are written together: 4 KB runs of the head-major output.
#include "bsa_device.cuh"
#include "bsa_kernels.h"

namespace bsa {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;   // rows a CTA holds at a time
constexpr int kUnroll = 4;             // rows in flight per 16-lane group

template <class T>
struct Raw8;                           // 8 elements as loaded
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
};
template <>
struct Raw8<float> {
  float4 a, b;
};

__device__ __forceinline__ uint4 ld_row16(const void* p) {
  uint4 r;
  // not the read-only path: in place, this call's own stores hit the same rows
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw8<__nv_bfloat16>& r) {
  r.v = ld_row16(p);
}
__device__ __forceinline__ void load8(const float* p, Raw8<float>& r) {
  const uint4 a = ld_row16(p), b = ld_row16(p + 4);
  r.a = *reinterpret_cast<const float4*>(&a);
  r.b = *reinterpret_cast<const float4*>(&b);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float x[8]) {
  bf16x8_to_f32(r.v, x);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float x[8]) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
  x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
// fp32 values, rounded once to the output type (to nearest even)
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float x[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float x[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <class Tin, class Tout>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  __shared__ float xch[kRows][kDim];   // partner exchange of the unaligned halves layout
  const int lane16 = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int ntens = a.ntens;
  const int b = blockIdx.z / ntens, t = blockIdx.z % ntens;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * a.tt + (group & (a.tt - 1));
  const int hstep = kRows / a.tt;
  const int h_end = min(a.H, static_cast<int>(blockIdx.y + 1) * a.hchunk);
  const int h0 = blockIdx.y * a.hchunk + group / a.tt;
  const bool live = n < a.N;
  const int e0 = lane16 * 8;
  const int r = a.turn[t] ? a.r : 0, half = r >> 1;
  const bool norm = a.weight[t] != nullptr;

  // cos and sin of this lane's 8 dimensions; sin carries the pair's sign
  float c[8], s[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f, w[j] = 1.f;
  if (live && e0 < r) {
    const int32_t* pos = a.positions + b * a.pos_b + n * a.pos_n;
    auto turn = [&](int i, float* sn, float* cs) {
      int axis = 0;
      while (i >= a.axis_end[axis]) ++axis;
      const double f = __ldg(a.freqs + i) * 0.15915494309189533577;   // turns a position
      const int64_t step = __double2ll_rn((f - rint(f)) * 18446744073709551616.0);
      const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(step) *
                                                 static_cast<uint64_t>(static_cast<int64_t>(pos[axis])));
      // [-2^31, 2^31) of a turn in 2^-32 units -> half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, sn, cs);
    };
    if (a.interleaved) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if (e0 + j < r) {
          float sn, cs;
          turn((e0 + j) >> 1, &sn, &cs);
          c[j] = c[j + 1] = cs * a.scale;
          s[j + 1] = sn * a.sin_scale;
          s[j] = -s[j + 1];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        if (e < r) {
          float sn, cs;
          turn(e < half ? e : e - half, &sn, &cs);
          c[j] = cs * a.scale;
          s[j] = (e < half ? -sn : sn) * a.sin_scale;
        }
      }
    }
  }
  if (norm) {
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.weight[t] + e0));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(a.weight[t] + e0 + 4));
    w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w;
    w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
  }

  const Tin* src = static_cast<const Tin*>(a.in[t]) + b * a.in_b + n * a.in_n + e0;
  Tout* dst = static_cast<Tout*>(a.out[t]) + b * a.out_b + n * a.out_n + e0;
  // all lanes of a warp walk the same number of steps (the shuffles need them)
  for (int hb = h0 - group / a.tt; hb < h_end; hb += hstep * kUnroll) {
    Raw8<Tin> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + group / a.tt + u * hstep;
      if (live && h < h_end) load8(src + h * a.in_h, raw[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (hb + u * hstep >= h_end) break;            // the same for the whole CTA
      const int h = hb + group / a.tt + u * hstep;
      const bool on = live && h < h_end;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
      if (on) unpack8(raw[u], x);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = rsqrtf(ss * (1.f / kDim) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * rs * w[j];
      }
      if (r > 0) {
        float y[8];
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
        } else if ((r & 15) == 0) {                  // partners sit r / 16 lanes away
          const int from = (lane16 * 8 < half) ? lane16 + (r >> 4) : lane16 - (r >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from & 15, 16);
        } else {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) xch[group][e0 + j] = x[j];
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = e0 + j;
            y[j] = xch[group][e < half ? e + half : (e < r ? e - half : e)];
          }
        }
        // dimensions past r pass unchanged (a 0 * infinity there would be NaN)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j < r) x[j] = fmaf(y[j], s[j], x[j] * c[j]);
      }
      if (on) store8(dst + h * a.out_h, x);
    }
  }
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, int in_fp32, int out_fp32, cudaStream_t st) {
  int tt = 1;
  while (tt < kRows && tt < a.N) tt *= 2;
  a.tt = tt;
  const int hstep = kRows / tt;
  const int64_t tiles = (static_cast<int64_t>(a.N) + tt - 1) / tt * a.B * a.ntens;
  // Split the heads until every SM has its eight CTAs; more would only repeat
  // the angles.
  const int64_t want = 148 * 8;
  int64_t chunks = (want + tiles - 1) / tiles;
  const int most = (a.H + hstep - 1) / hstep;
  if (chunks > most) chunks = most;
  a.hchunk = (a.H + static_cast<int>(chunks) - 1) / static_cast<int>(chunks);
  a.hchunk = (a.hchunk + hstep - 1) / hstep * hstep;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.N) + tt - 1) / tt),
                  (a.H + a.hchunk - 1) / a.hchunk, a.B * a.ntens);
  using bf16 = __nv_bfloat16;
  if (in_fp32 && out_fp32)
    rotary_kernel<float, float><<<grid, kThreads, 0, st>>>(a);
  else if (in_fp32)
    rotary_kernel<float, bf16><<<grid, kThreads, 0, st>>>(a);
  else if (out_fp32)
    rotary_kernel<bf16, float><<<grid, kThreads, 0, st>>>(a);
  else
    rotary_kernel<bf16, bf16><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace bsa
