// Rows to int8 codes with one scale a row (rows.cuh: store_codes), the left
// operand of the int8 product and, once, its weights.
//
// Row (b, n) has S segments of L values; segment s starts at b x_b + n x_n +
// s x_s.  The attention's head-major output [B, H, N, 128] is read as token
// rows of H segments of 128, so no transposed copy is made.  HBM-bound: each
// value is read once (2 B) and its code written once (1 B).
#include "bsa_kernels.h"
#include "rows.cuh"

namespace bsa {

namespace {

template <class Tx, int CH, int kThreads, bool kVec>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) quant_int8_kernel(const QuantInt8Args a) {
  __shared__ RowReduce red;
  RowGroup g{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 0, &red, 0};
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  const int n = a.S * a.L;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = row / a.N, t = row - b * a.N;
    const Tx* src = static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n;
    float x[CH][8];
    if (a.S == 1) {
      load_row<CH, kVec>(g, src, n, x);
    } else {
      if constexpr (kVec) {       // L is a multiple of 8: a chunk lies in one segment
        constexpr int W = static_cast<int>(sizeof(Tx)) / 2;   // 16-byte words a chunk
        uint4 w[CH][W];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = row_index<true>(g, c, 0);
          const int s = i / a.L;
#pragma unroll
          for (int k = 0; k < W; ++k) {
            w[c][k] = make_uint4(0, 0, 0, 0);
            if (i < n) w[c][k] = ld_row_v4(src + s * a.x_s + (i - s * a.L) + 4 * k);
          }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if constexpr (W == 1) {
            bf16x8_to_f32(w[c][0], x[c]);
          } else {
#pragma unroll
            for (int k = 0; k < W; ++k) {
              x[c][4 * k] = __uint_as_float(w[c][k].x), x[c][4 * k + 1] = __uint_as_float(w[c][k].y);
              x[c][4 * k + 2] = __uint_as_float(w[c][k].z), x[c][4 * k + 3] = __uint_as_float(w[c][k].w);
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int i = row_index<false>(g, c, j);
            const int s = i / a.L;
            x[c][j] = i < n ? to_f32(src[s * a.x_s + (i - s * a.L)]) : 0.f;
          }
      }
    }
    const float s = store_codes<CH, kVec>(g, x, n, a.q + row * a.q_ld);
    if (threadIdx.x == 0) a.scale[row] = s;
  }
}

template <class Tx, bool kVec>
cudaError_t launch(const QuantInt8Args& a, int ch, int threads, int blocks, cudaStream_t st) {
  auto go = [&](auto k) {
    k<<<blocks, threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (ch == 1) return go(quant_int8_kernel<Tx, 1, 1024, kVec>);
  if (ch == 2) return go(quant_int8_kernel<Tx, 2, 1024, kVec>);
  if (threads <= 256) return go(quant_int8_kernel<Tx, 4, 256, kVec>);
  if (threads <= 512) return go(quant_int8_kernel<Tx, 4, 512, kVec>);
  return go(quant_int8_kernel<Tx, 4, 1024, kVec>);
}

}  // namespace

cudaError_t launch_quant_int8(const QuantInt8Args& a, bool x_fp32, bool vec, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  int ch, threads;
  row_shape(a.S * a.L, rows, &ch, &threads);
  const int blocks = static_cast<int>(rows < (1 << 30) ? rows : (1 << 30));
  if (vec)
    return x_fp32 ? launch<float, true>(a, ch, threads, blocks, st)
                  : launch<__nv_bfloat16, true>(a, ch, threads, blocks, st);
  return x_fp32 ? launch<float, false>(a, ch, threads, blocks, st)
                : launch<__nv_bfloat16, false>(a, ch, threads, blocks, st);
}

}  // namespace bsa
