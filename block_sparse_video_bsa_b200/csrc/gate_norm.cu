// Norms before and after a block, fused with its gate and residual: for every
// row of C values
//   h = residual_scale x + branch_scale gate * post(y)   (x alone without y)
//   z = pre(h) (1 + scale) + shift
// post and pre each nothing, an RMS norm or a layer norm with optional weight
// and bias; gate, scale and shift one vector a batch entry, or one a token.  z
// as bf16 or fp32, or as int8 codes with one scale a row for the projection
// that follows.
//
// HBM-bound: x and y are read once and h and z written once; a row stays in
// registers between its sums.  All sums and statistics are fp32, z is formed
// from the unrounded h.  The vectors that rows share come from L1 / L2.
#include "bsa_kernels.h"
#include "rows.cuh"

namespace bsa {

namespace {

// v = norm(v) * weight + bias, in registers
template <int CH, bool kVec>
__device__ __forceinline__ void norm_row(float (&v)[CH][8], int n, int kind, float eps,
                                         const float* weight, const float* bias, RowReduce& red,
                                         int& turn) {
  if (kind == kNormLayer) {
    const float2 mv = row_moments<CH, kVec>(v, n, red, turn);
    const float rs = rsqrtf(mv.y + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = (v[c][j] - mv.x) * rs;
  } else if (kind == kNormRms) {
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(v[c][j], v[c][j], q);   // 0 past n
    const float rs = rsqrtf(row_sum(q, red, turn) / n + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= rs;
  }
  if (weight) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kVec>(weight, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= w[j];
    }
  }
  if (bias) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kVec>(bias, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] += w[j];
    }
  }
}

template <bool kVec>
__device__ __forceinline__ void load_mod8(const void* p, int fp32, int64_t off, int n, int c,
                                          float v[8]) {
  if (fp32)
    load_shared8<kVec>(static_cast<const float*>(p) + off, n, c, v);
  else
    load_shared8<kVec>(static_cast<const __nv_bfloat16*>(p) + off, n, c, v);
}

template <class Tx, int CH, int kThreads, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) gate_norm_kernel(const GateNormArgs a) {
  __shared__ RowReduce red;
  int turn = 0;
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = row / a.N, t = row - b * a.N;
    float h[CH][8];
    load_row<CH, kVec>(static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n, a.C, h);
    if (a.y) {
      float y[CH][8];
      if (a.y_fp32)
        load_row<CH, kVec>(static_cast<const float*>(a.y) + b * a.y_b + t * a.y_n, a.C, y);
      else
        load_row<CH, kVec>(static_cast<const __nv_bfloat16*>(a.y) + b * a.y_b + t * a.y_n, a.C, y);
      norm_row<CH, kVec>(y, a.C, a.post, a.eps, a.post_weight, a.post_bias, red, turn);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (a.gate) {
          float g[8];
          load_mod8<kVec>(a.gate, a.mod_fp32, b * a.gate_b + t * a.gate_n, a.C, c, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[c][j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[c][j] = fmaf(y[c][j], a.branch_scale, h[c][j] * a.residual_scale);
          if (row_index<kVec>(c, j) >= a.C) h[c][j] = 0.f;   // a bias reached past the row
        }
        if (a.h) store8<kVec>(static_cast<Tx*>(a.h) + b * a.h_b + t * a.h_n, a.C, c, h[c]);
      }
    }
    if (!a.z) continue;
    norm_row<CH, kVec>(h, a.C, a.pre, a.eps, a.pre_weight, a.pre_bias, red, turn);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.mscale) {
        float g[8];
        load_mod8<kVec>(a.mscale, a.mod_fp32, b * a.scale_b + t * a.scale_n, a.C, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = fmaf(h[c][j], g[j], h[c][j]);
      }
      if (a.shift) {
        float g[8];
        load_mod8<kVec>(a.shift, a.mod_fp32, b * a.shift_b + t * a.shift_n, a.C, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += g[j];
      }
      const int64_t o = b * a.z_b + t * a.z_n;
      if (a.z_type == kTypeBf16)
        store8<kVec>(static_cast<__nv_bfloat16*>(a.z) + o, a.C, c, h[c]);
      else if (a.z_type == kTypeFp32)
        store8<kVec>(static_cast<float*>(a.z) + o, a.C, c, h[c]);
    }
    if (a.z_type == kTypeInt8) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row_index<kVec>(c, j) >= a.C) h[c][j] = 0.f;   // a layer norm's mean reached past the row
      const float s = store_codes<CH, kVec>(h, a.C, static_cast<int8_t*>(a.z) + b * a.z_b + t * a.z_n,
                                            red, turn);
      if (threadIdx.x == 0) a.z_scale[row] = s;
    }
  }
}

template <class Tx, bool kVec>
cudaError_t launch(const GateNormArgs& a, int ch, int threads, int blocks, cudaStream_t st) {
  auto go = [&](auto k) {
    k<<<blocks, threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (ch == 1) return go(gate_norm_kernel<Tx, 1, 1024, kVec>);
  if (ch == 2) return go(gate_norm_kernel<Tx, 2, 1024, kVec>);
  if (threads <= 256) return go(gate_norm_kernel<Tx, 4, 256, kVec>);
  if (threads <= 512) return go(gate_norm_kernel<Tx, 4, 512, kVec>);
  return go(gate_norm_kernel<Tx, 4, 1024, kVec>);
}

}  // namespace

// Threads and chunks (1, 2 or 4) of a row of n <= 32,768 values: four chunks a
// thread, fewer for short rows and for few rows, where a row's latency counts.
void row_shape(int n, int64_t rows, int* ch, int* threads) {
  const int vecs = (n + 7) / 8;
  int c = rows >= 148 * 2 ? 4 : 1;
  while (c > 1 && (vecs + c - 1) / c < 32) c /= 2;
  while ((vecs + c - 1) / c > 1024) c *= 2;
  *ch = c;
  *threads = ((vecs + c - 1) / c + 31) / 32 * 32;
}

cudaError_t launch_gate_norm(const GateNormArgs& a, bool x_fp32, bool vec, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  int ch, threads;
  row_shape(a.C, rows, &ch, &threads);
  const int blocks = static_cast<int>(rows < (1 << 30) ? rows : (1 << 30));
  if (vec)
    return x_fp32 ? launch<float, true>(a, ch, threads, blocks, st)
                  : launch<__nv_bfloat16, true>(a, ch, threads, blocks, st);
  return x_fp32 ? launch<float, false>(a, ch, threads, blocks, st)
                : launch<__nv_bfloat16, false>(a, ch, threads, blocks, st);
}

}  // namespace bsa
