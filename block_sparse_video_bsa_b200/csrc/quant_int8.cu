// Rows to int8 codes with one scale a row (rows.cuh: store_codes), the left
// operand of the int8 product and, once, its weights.  |code| <= 127.
//
// Row (b, n) has S segments of L values; segment s starts at b x_b + n x_n +
// s x_s.  The attention's head-major output [B, H, N, 128] is read as token
// rows of H segments of 128, so no transposed copy is made.  HBM-bound: each
// value is read once (2 B) and its code written once (1 B); 130 us for
// 37,740 x 7,168 head-major bf16, 127 us for rows, 6.2 and 6.4 TB/s.  Rows off
// 16 bytes go value by value (20,000 x 3,971 bf16: 158 us, 1.5 TB/s).
#include "bsa_kernels.h"
#include "rows.cuh"

namespace bsa {

namespace {

// Any rows, fp32 in registers.
template <class Tx, int CH, int kMode>
__global__ void __launch_bounds__(1024, 1) quant_int8_kernel(const QuantInt8Args a) {
  grid_wait();
  grid_ready();
  __shared__ RowReduce red;
  RowGroup g{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 0, &red, 0, 0};
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  const int n = a.S * a.L;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = row / a.N, t = row - b * a.N;
    const Tx* src = static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n;
    float x[CH][8];
    if (a.S == 1) {
      load_row<CH, kMode>(g, src, n, x);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = row_index<kMode>(g, c, j);
          const int s = i / a.L;
          x[c][j] = i < n ? to_f32(src[s * a.x_s + (i - s * a.L)]) : 0.f;
        }
    }
    const float s = store_codes<CH, kMode>(g, x, n, a.q + row * a.q_ld);
    if (g.tid == 0) a.scale[row] = s;
  }
}

// bf16 rows of aligned 8-value chunks: the words stay packed between the two
// steps (half the registers, so more rows in flight on an SM), and the maximum
// is taken on them as 16-bit integers, which order magnitudes with NaN on top.
template <int CH, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) quant_int8_bf16_kernel(const QuantInt8Args a) {
  grid_wait();
  grid_ready();
  __shared__ RowReduce red;
  RowGroup g{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 0, &red, 0, 0};
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  const int n = a.S * a.L;
  int64_t off[CH];                               // of this thread's chunks in every row
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = row_index<kAligned>(g, c, 0);
    const int s = a.S == 1 ? 0 : i / a.L;        // a chunk lies in one segment
    off[c] = s * a.x_s + (i - s * a.L);
  }
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = a.B == 1 ? 0 : row / a.N, t = row - b * a.N;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.x) + b * a.x_b + t * a.x_n;
    uint4 w[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      w[c] = make_uint4(0, 0, 0, 0);
      if (row_index<kAligned>(g, c, 0) < n) w[c] = ld_row_v4(src + off[c]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      m = __vmaxu2(m, __vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu));
    }
    const uint32_t top = max(m & 0xffffu, m >> 16) << 16;
    float am = row_max_abs(g, __uint_as_float(top));
    const bool finite = am <= 3.402823466e38f;
    am = finite ? fmaxf(am, kInt8Floor) : am;
    const float inv = __fdiv_rn(127.f, am);
    int8_t* q = a.q + row * a.q_ld;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = row_index<kAligned>(g, c, 0);
      float x[8];
      bf16x8_to_f32(w[c], x);
      uint2 k = make_uint2(0, 0);
      if (finite) k = make_uint2(codes4(x, inv), codes4(x + 4, inv));
      if (i < n) *reinterpret_cast<uint2*>(q + i) = k;
    }
    if (g.tid == 0) a.scale[row] = finite ? __fdiv_rn(am, 127.f) : __uint_as_float(0x7fc00000u);
  }
}

template <class Tx, int kMode>
cudaError_t launch(const QuantInt8Args& a, int ch, int threads, int blocks, cudaStream_t st) {
  auto go = [&](auto k) {
    return launch_early(k, dim3(blocks), threads, 0, st, 0, a);
  };
  if (ch == 1) return go(quant_int8_kernel<Tx, 1, kMode>);
  if (ch == 2) return go(quant_int8_kernel<Tx, 2, kMode>);
  return go(quant_int8_kernel<Tx, 4, kMode>);
}

}  // namespace

cudaError_t launch_quant_int8(const QuantInt8Args& a, bool x_fp32, bool vec, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  int ch, threads;
  row_shape(a.S * a.L, rows, 2 * 148, &ch, &threads);
  int blocks = static_cast<int>(rows < (1 << 30) ? rows : (1 << 30));
  if (vec && !x_fp32) {
    const int vecs = (a.S * a.L + 7) / 8;
    if (ch > 1) {
      ch = 4;
      threads = ((vecs + 3) / 4 + 31) / 32 * 32;
      // as many CTAs as are resident at once: 131 us for 37,740 head-major rows of 7,168 against
      // 142 with a CTA a row
      const int resident = 1536 / threads < 32 ? 1536 / threads : 32;
      if (resident > 0 && blocks > 148 * resident) blocks = 148 * resident;
    }
    auto go = [&](auto k) {
      return launch_early(k, dim3(blocks), threads, 0, st, 0, a);
    };
    if (ch == 1) return go(quant_int8_bf16_kernel<1, 1024, 1>);
    if (threads <= 256) return go(quant_int8_bf16_kernel<4, 256, 6>);
    return go(quant_int8_bf16_kernel<4, 1024, 1>);
  }
  if (vec) return launch<float, kAligned>(a, ch, threads, blocks, st);
  return x_fp32 ? launch<float, kSingles>(a, ch, threads, blocks, st)
                : launch<__nv_bfloat16, kSingles>(a, ch, threads, blocks, st);
}

}  // namespace bsa
