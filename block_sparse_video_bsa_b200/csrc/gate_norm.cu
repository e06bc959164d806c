// Norms before and after a block, fused with its gate and residual: for every
// row of C values
//   h = residual_scale x + branch_scale gate * post(y)   (x alone without y)
//   z = pre(h) (1 + scale) + shift
// post and pre each nothing, an RMS norm or a layer norm with optional weight
// and bias; gate, scale and shift one vector a batch entry, or one a token.  z
// as bf16 or fp32, or as int8 codes with one scale a row for the projection
// that follows.
//
// HBM-bound: x and y are read once and h and z written once.  All sums and
// statistics are fp32, z is formed from the unrounded h.
//
// Two kernels.  gate_norm_ring_kernel for many aligned rows: one CTA per SM
// keeps the vectors folded together in shared memory (three or four loads a row
// saved), a producer warp streams rows, and vectors with an entry a token,
// through a ring of shared-memory stages with bulk copies, and several groups
// of warps each take the next row, so that the loads in flight do not depend on
// registers and one group's reductions hide behind another's work (37,740 x
// 7,168 bf16, layer and RMS norm: 365 to 399 us, 5.4 to 5.9 TB/s; a CTA a row
// takes 650 us; RMS norm to codes 223 us, 3.6 TB/s, where the folded vectors
// from shared memory and two reductions a row are most of the work for three
// bytes a value).  Short rows come several a stage.  gate_norm_kernel for the rest: one CTA a
// row, the row in registers between its sums, the vectors from L1 / L2; odd
// rows in shifted chunks (20,000 x 3,971: 280 us, 2.3 TB/s; value by value
// 850).
#include <type_traits>

#include "bsa_kernels.h"
#include "rows.cuh"

namespace bsa {

namespace {

// ------------------------------------------------------------ one CTA a row

// v = norm(v) * weight + bias, in registers
template <int CH, int kMode>
__device__ __forceinline__ void norm_row(RowGroup& g, float (&v)[CH][8], int n, int kind, float eps,
                                         const float* weight, const float* bias) {
  if (kind == kNormLayer) {
    const float2 mv = row_moments<CH, kMode>(g, v, n);
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
    const float rs = rsqrtf(__fadd_rn(row_mean(g, q, n), eps));
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= rs;
  }
  if (weight) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kMode>(g, weight, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= w[j];
    }
  }
  if (bias) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kMode>(g, bias, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] += w[j];
    }
  }
}

// A chunk of gate, scale or shift: one vector a token lies as the rows do.
template <int kMode>
__device__ __forceinline__ void load_mod8(const RowGroup& g, const void* p, int fp32, int64_t off,
                                          bool token, int n, int c, float v[8]) {
  const float* f = static_cast<const float*>(p) + off;
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p) + off;
  if (kMode == kShifted && token && row_whole<kMode>(g, c, n)) {
    if (fp32)
      chunk_words(f + row_index<kMode>(g, c, 0), v);
    else
      chunk_words(h + row_index<kMode>(g, c, 0), v);
  } else if (fp32) {
    load_shared8<kMode>(g, f, n, c, v);
  } else {
    load_shared8<kMode>(g, h, n, c, v);
  }
}

template <int kMode>
__device__ __forceinline__ void store_z8(const RowGroup& g, const GateNormArgs& a, int64_t o, int c,
                                         const float v[8]) {
  if (a.z_type == kTypeBf16)
    store8<kMode>(g, static_cast<__nv_bfloat16*>(a.z) + o, a.C, c, v);
  else if (a.z_type == kTypeFp32)
    store8<kMode>(g, static_cast<float*>(a.z) + o, a.C, c, v);
}

template <class Tx, int CH, int kThreads, int kBlocks, int kMode>
__global__ void __launch_bounds__(kThreads, kBlocks) gate_norm_kernel(const GateNormArgs a) {
  grid_wait();
  grid_ready();
  __shared__ RowReduce red;
  RowGroup g{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 0, &red, 0, 0};
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = a.B == 1 ? 0 : row / a.N, t = row - b * a.N;
    if (kMode == kShifted) g.shift = static_cast<int>((b * a.x_b + t * a.x_n) & 7);
    float h[CH][8];
    load_row<CH, kMode>(g, static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n, a.C, h);
    // with one chunk a thread there is room to have the vectors under way with the row
    constexpr bool kEarly = CH == 1;
    float mg[8], ms[8], mt[8];
    if (kEarly) {
      if (a.gate) load_mod8<kMode>(g, a.gate, a.mod_fp32, b * a.gate_b + t * a.gate_n, a.gate_n != 0, a.C, 0, mg);
      if (a.mscale) load_mod8<kMode>(g, a.mscale, a.mod_fp32, b * a.scale_b + t * a.scale_n, a.scale_n != 0, a.C, 0, ms);
      if (a.shift) load_mod8<kMode>(g, a.shift, a.mod_fp32, b * a.shift_b + t * a.shift_n, a.shift_n != 0, a.C, 0, mt);
    }
    if (a.y) {
      float y[CH][8];
      const int64_t o = b * a.y_b + t * a.y_n;
      if (a.y_fp32)
        load_row<CH, kMode>(g, static_cast<const float*>(a.y) + o, a.C, y);
      else
        load_row<CH, kMode>(g, static_cast<const __nv_bfloat16*>(a.y) + o, a.C, y);
      norm_row<CH, kMode>(g, y, a.C, a.post, a.eps, a.post_weight, a.post_bias);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (a.gate) {
          float m[8];
          if (!kEarly)
            load_mod8<kMode>(g, a.gate, a.mod_fp32, b * a.gate_b + t * a.gate_n, a.gate_n != 0, a.C, c, m);
          else
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = mg[j];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[c][j] *= m[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[c][j] = fmaf(y[c][j], a.branch_scale, h[c][j] * a.residual_scale);
          if (!row_in<kMode>(g, c, j, a.C)) h[c][j] = 0.f;   // a norm reached past the row
        }
        if (a.h) store8<kMode>(g, static_cast<Tx*>(a.h) + b * a.h_b + t * a.h_n, a.C, c, h[c]);
      }
    }
    if (!a.z) continue;
    norm_row<CH, kMode>(g, h, a.C, a.pre, a.eps, a.pre_weight, a.pre_bias);
    const int64_t o = b * a.z_b + t * a.z_n;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.mscale) {
        float m[8];
        if (!kEarly)
          load_mod8<kMode>(g, a.mscale, a.mod_fp32, b * a.scale_b + t * a.scale_n, a.scale_n != 0, a.C, c, m);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) m[j] = ms[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = __fmul_rn(h[c][j], __fadd_rn(1.f, m[j]));
      }
      if (a.shift) {
        float m[8];
        if (!kEarly)
          load_mod8<kMode>(g, a.shift, a.mod_fp32, b * a.shift_b + t * a.shift_n, a.shift_n != 0, a.C, c, m);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) m[j] = mt[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = __fadd_rn(h[c][j], m[j]);
      }
      store_z8<kMode>(g, a, o, c, h[c]);
    }
    if (a.z_type == kTypeInt8) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!row_in<kMode>(g, c, j, a.C)) h[c][j] = 0.f;   // a layer norm's mean reached past the row
      const float s = store_codes<CH, kMode>(g, h, a.C, static_cast<int8_t*>(a.z) + o);
      if (g.tid == 0) a.z_scale[row] = s;
    }
  }
}

// ------------------------------------------------------------ rows through a ring

constexpr int kRingThreads = 704;      // 21 warps of rows at most, and the producer warp
constexpr int kMaxGroups = 15;         // named barriers; groups of one warp need none
constexpr int kMaxStages = 24;
constexpr uint32_t kRingSmem = 227 * 1024;

struct RingCtl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort_flag;
};

// What shared memory holds, in floats and bytes.
struct RingShape {
  int threads, groups, stages;   // threads of a group
  int rows, log_rows;            // rows a stage: one copy brings them where they are contiguous
  int has_gain, has_post_bias;   // gate * post_weight, gate * post_bias
  int has_a, has_b;              // pre_weight (1 + scale), pre_bias (1 + scale) + shift
  int tok_gate, tok_mod;         // gate, scale and shift with a vector a token: streamed with the rows
  uint32_t m_bytes, gate_at, scale_at, shift_at;   // of such a vector; where a stage has them
  uint32_t x_bytes, y_bytes;     // of a row
  uint32_t row_bytes;            // of a row and the vectors that come with it
  uint32_t stage_bytes, y_at;    // of a stage; where its rows of y start
  uint32_t off_stage, off_red, off_ctl, bytes;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// This thread has read its part of a stage.  The next filling comes through the
// async proxy, which does not wait for reads of the generic one by itself: the
// fence orders them before the arrival.
__device__ __forceinline__ void stage_read(uint64_t* empty) {
  fence_proxy_async_smem();
  mbar_arrive(empty);
}

// 8 values as four pairs: the packed fp32 instructions halve the arithmetic,
// which is what bounds this kernel next to HBM.
struct Oct {
  float2 p[4];
};
// max(|a|, |b|, m), NaN if one of them is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float m) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(m));
  return d;
}
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

__device__ __forceinline__ void smem8(const __nv_bfloat16* p, Oct& v) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v.p[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
}
__device__ __forceinline__ void smem8(const float* p, Oct& v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v.p[0] = make_float2(a.x, a.y), v.p[1] = make_float2(a.z, a.w);
  v.p[2] = make_float2(b.x, b.y), v.p[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ void smem8_mod(const uint8_t* p, int fp32, int i, Oct& v) {
  if (fp32)
    smem8(reinterpret_cast<const float*>(p) + i, v);
  else
    smem8(reinterpret_cast<const __nv_bfloat16*>(p) + i, v);
}

// A vector folded in shared memory: the 8 values of 32 neighbouring threads
// are kept as their first fours, then their second fours, so that a warp's
// 16-byte loads meet every bank once.  at: where value i lies; load: chunk k / 8.
__device__ __forceinline__ int folded_at(int i) {
  return (i & ~255) | ((i & 4) << 5) | ((i & 248) >> 1) | (i & 3);
}
__device__ __forceinline__ void folded8(const float* p, int k, Oct& v) {
  const int at = folded_at(k);
  const float4 a = *reinterpret_cast<const float4*>(p + at);
  const float4 b = *reinterpret_cast<const float4*>(p + at + 128);
  v.p[0] = make_float2(a.x, a.y), v.p[1] = make_float2(a.z, a.w);
  v.p[2] = make_float2(b.x, b.y), v.p[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ void put8(__nv_bfloat16* p, const Oct& v) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v.p[0].x, v.p[0].y), pack_bf16x2(v.p[1].x, v.p[1].y),
                 pack_bf16x2(v.p[2].x, v.p[2].y), pack_bf16x2(v.p[3].x, v.p[3].y));
}
__device__ __forceinline__ void put8(float* p, const Oct& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
}

// (m, r) with norm(v) = v r + m for a row that `get` gives chunk by chunk;
// in[c]: the chunk lies inside the row (the others are copies of its last);
// cnt: values of the row that the warp holds, and its reciprocal (0 for none).
template <int CH, class Get>
__device__ __forceinline__ float2 row_affine(RowGroup& g, int n, int kind, float eps,
                                             const bool (&in)[CH], float cnt, float inv_cnt,
                                             Get get) {
  if (kind == kNormNone) return make_float2(0.f, 1.f);
  if (kind == kNormRms) {
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      Oct v;
      get(c, v);
      float2 s = mul2(v.p[0], v.p[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) s = fma2(v.p[j], v.p[j], s);
      q += in[c] ? s.x + s.y : 0.f;
    }
    return make_float2(0.f, rsqrtf(__fadd_rn(row_mean(g, q, n), eps)));
  }
  // as row_moments (rows.cuh)
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Oct v;
    get(c, v);
    const float2 t = add2(add2(v.p[0], v.p[1]), add2(v.p[2], v.p[3]));
    s += in[c] ? t.x + t.y : 0.f;
  }
  const float mean = warp_sum(s) * inv_cnt;
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Oct v;
    get(c, v);
    float2 d = add2(v.p[0], pair(-mean));
    float2 t = mul2(d, d);
#pragma unroll
    for (int j = 1; j < 4; ++j) {
      d = add2(v.p[j], pair(-mean));
      t = fma2(d, d, t);
    }
    q += in[c] ? t.x + t.y : 0.f;
  }
  const float2 mv = combine_moments(g, mean, warp_sum(q), cnt, n);
  const float r = rsqrtf(mv.y + eps);
  const float m = -mv.x * r;
  // m past fp32 with a finite r: a deviation is 2^-24 of the mean at least, which
  // would hold |m| below 2^24 sqrt(n), so there is none and the norm is 0
  if (fabsf(m) == INFINITY && r < INFINITY) return make_float2(0.f, 0.f);
  return make_float2(m, r);
}

template <class Tx, class Ty, int CH>
__global__ void __launch_bounds__(kRingThreads, 1) gate_norm_ring_kernel(const GateNormArgs a,
                                                                        const RingShape s) {
  extern __shared__ __align__(128) uint8_t sm[];
  RingCtl* ctl = reinterpret_cast<RingCtl*>(sm + s.off_ctl);
  const int rows_threads = s.groups * s.threads;
  const int64_t b = blockIdx.y;
  const int C = a.C;
  const int len = (C + 255) & ~255;                                // of a folded vector
  float* gain = reinterpret_cast<float*>(sm);                      // branch_scale gate post_weight
  float* pbias = gain + (s.has_gain ? len : 0);                    // branch_scale gate post_bias
  float* va = pbias + (s.has_post_bias ? len : 0);                 // pre_weight (1 + scale)
  float* vb = va + (s.has_a ? len : 0);                            // pre_bias (1 + scale) + shift
  if (threadIdx.x == 0) {
    for (int i = 0; i < s.stages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], s.rows * s.threads);
    }
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_wait();
  grid_ready();
  const WaitCtx wc{&ctl->abort_flag, a.dev_status};
  // the CTA's rows in turn: s.rows neighbours of every gridDim.x-th block of them
  const int blocks = (a.N + s.rows - 1) / s.rows;

  if (static_cast<int>(threadIdx.x) >= rows_threads) {
    if (static_cast<int>(threadIdx.x) == rows_threads) {
      uint32_t st = 0, round = 0;
      for (int q = blockIdx.x; q < blocks; q += gridDim.x) {
        if (round > 0 && !mbar_wait(&ctl->empty[st], (round - 1) & 1, wc)) break;
        const int64_t t = static_cast<int64_t>(q) * s.rows;
        const uint32_t n = static_cast<uint32_t>(a.N - t < s.rows ? a.N - t : s.rows);
        uint8_t* dst = sm + s.off_stage + st * s.stage_bytes;
        mbar_arrive_expect_tx(&ctl->full[st], n * s.row_bytes);
        bulk_load(dst, static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n, n * s.x_bytes,
                  &ctl->full[st]);
        if (s.y_bytes)
          bulk_load(dst + s.y_at, static_cast<const Ty*>(a.y) + b * a.y_b + t * a.y_n,
                    n * s.y_bytes, &ctl->full[st]);
        auto vector = [&](uint32_t at, const void* p, int64_t o) {
          bulk_load(dst + at, static_cast<const char*>(p) + o * (a.mod_fp32 ? 4 : 2), n * s.m_bytes,
                    &ctl->full[st]);
        };
        if (s.tok_gate) vector(s.gate_at, a.gate, b * a.gate_b + t * a.gate_n);
        if (s.tok_mod && a.mscale) vector(s.scale_at, a.mscale, b * a.scale_b + t * a.scale_n);
        if (s.tok_mod && a.shift) vector(s.shift_at, a.shift, b * a.shift_b + t * a.shift_n);
        if (++st == static_cast<uint32_t>(s.stages)) st = 0, ++round;
      }
      // every issued load has landed before the CTA exits
      for (int i = 0; i < s.stages; ++i) {
        if (round == 0 && st == 0) break;
        if (st == 0) st = s.stages, --round;
        --st;
        mbar_wait(&ctl->full[st], round & 1, wc);
      }
    }
    return;
  }

  {
    // the vectors, 8 values a thread
    auto mod = [&](const void* p, int64_t off, int i, float none, float v[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = none;
      if (!p) return;
      if (a.mod_fp32)
        chunk_words(static_cast<const float*>(p) + off + i, v);
      else
        chunk_words(static_cast<const __nv_bfloat16*>(p) + off + i, v);
    };
    auto put = [&](float* p, int i, const float v[8]) {
      float4* q = reinterpret_cast<float4*>(p + folded_at(i));
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[32] = make_float4(v[4], v[5], v[6], v[7]);
    };
    for (int i = 8 * threadIdx.x; i < C; i += 8 * rows_threads) {
      float gt[8], sc[8], sh[8], w[8], o[8];
      mod(s.tok_gate ? nullptr : a.gate, b * a.gate_b, i, 1.f, gt);
      mod(s.tok_mod ? nullptr : a.mscale, b * a.scale_b, i, 0.f, sc);
      mod(s.tok_mod ? nullptr : a.shift, b * a.shift_b, i, 0.f, sh);
#pragma unroll
      for (int j = 0; j < 8; ++j) gt[j] *= a.branch_scale, sc[j] += 1.f, w[j] = 1.f;
      if (s.has_gain) {
        if (a.post_weight) chunk_words(a.post_weight + i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = gt[j] * w[j];
        put(gain, i, o);
      }
      if (s.has_post_bias) {
        chunk_words(a.post_bias + i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = gt[j] * w[j];
        put(pbias, i, o);
      }
      if (s.has_a) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
        if (a.pre_weight) chunk_words(a.pre_weight + i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = sc[j] * w[j];
        put(va, i, o);
      }
      if (s.has_b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.f;
        if (a.pre_bias) chunk_words(a.pre_bias + i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(w[j], sc[j], sh[j]);
        put(vb, i, o);
      }
    }
  }
  const int group = threadIdx.x / s.threads;
  RowReduce* red = reinterpret_cast<RowReduce*>(sm + s.off_red) + group;
  if (threadIdx.x % s.threads == 0) red->no[0] = red->no[1] = 0;
  asm volatile("bar.sync 0, %0;" ::"r"(rows_threads) : "memory");   // the producer is on its way

  RowGroup g{static_cast<int>(threadIdx.x) - group * s.threads, s.threads, 1 + group, red,
             0, 0};
  int mark = 0;
  // chunks past the row's end read its last one again and neither count nor store
  int at[CH];
  bool in[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = row_index<kAligned>(g, c, 0);
    in[c] = k < C;
    at[c] = in[c] ? k : C - 8;
  }
  float cnt = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) cnt += in[c] ? 8.f : 0.f;
  cnt = warp_sum(cnt);
  const float inv_cnt = cnt > 0.f ? 1.f / cnt : 0.f;
  // row `sub` of the CTA's stage number `seq`, stage seq % stages
  uint32_t sub = group % s.rows, st = group / s.rows, round = 0;
  int q = blockIdx.x + st * gridDim.x;
  while (st >= static_cast<uint32_t>(s.stages)) st -= s.stages, ++round;
  for (;;) {
    if (q >= blocks) break;
    const int64_t t = static_cast<int64_t>(q) * s.rows + sub;
    // A wait by parity tells a filling from the next one only: rows of a stage go
    // to different groups and loads land in any order, so this group first sees
    // that the stage's last filling was read (it was asked for before this group's
    // own last row, so its phase is the current one at most), then that this one
    // has landed.  The whole group goes on or none of it.
    const bool read = round == 0 || mbar_wait(&ctl->empty[st], (round - 1) & 1, wc);
    if (!g.all(read && mbar_wait(&ctl->full[st], round & 1, wc), mark)) break;
    const uint8_t* stage = sm + s.off_stage + st * s.stage_bytes;
    uint64_t* empty = &ctl->empty[st];
    const Tx* xs = reinterpret_cast<const Tx*>(stage + sub * s.x_bytes);
    const Ty* ys = reinterpret_cast<const Ty*>(stage + s.y_at + sub * s.y_bytes);
    const uint8_t* ms = stage + sub * s.m_bytes;
    sub += s.groups;
    const uint32_t on = sub >> s.log_rows;
    sub &= s.rows - 1;
    q += on * gridDim.x;
    for (st += on; st >= static_cast<uint32_t>(s.stages); st -= s.stages) ++round;
    if (t >= a.N) continue;             // past the last stage's rows
    Oct h[CH];
    if (s.y_bytes) {
      const float2 mr = row_affine<CH>(g, C, a.post, a.eps, in, cnt, inv_cnt,
                                       [&](int c, Oct& v) { smem8(ys + at[c], v); });
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        smem8(ys + at[c], h[c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c].p[j] = fma2(h[c].p[j], pair(mr.y), pair(mr.x));
      }
      if (s.has_gain) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Oct m;
          folded8(gain, at[c], m);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[c].p[j] = mul2(h[c].p[j], m.p[j]);
        }
      }
      if (s.has_post_bias) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Oct m;
          folded8(pbias, at[c], m);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[c].p[j] = add2(h[c].p[j], m.p[j]);
        }
      }
      if (s.tok_gate) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          Oct m;
          smem8_mod(ms + s.gate_at, a.mod_fp32, at[c], m);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[c].p[j] = mul2(h[c].p[j], m.p[j]);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Oct x;
        smem8(xs + at[c], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c].p[j] = fma2(x.p[j], pair(a.residual_scale), h[c].p[j]);
      }
      if (!s.tok_mod) stage_read(empty);
      if (a.h) {
        Tx* ho = static_cast<Tx*>(a.h) + b * a.h_b + t * a.h_n;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (in[c]) put8(ho + at[c], h[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) smem8(xs + at[c], h[c]);
      if (!s.tok_mod) stage_read(empty);
    }
    if (!a.z) continue;
    const float2 mr =
        row_affine<CH>(g, C, a.pre, a.eps, in, cnt, inv_cnt, [&](int c, Oct& v) { v = h[c]; });
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) h[c].p[j] = fma2(h[c].p[j], pair(mr.y), pair(mr.x));
    if (s.has_a) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Oct m;
        folded8(va, at[c], m);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c].p[j] = mul2(h[c].p[j], m.p[j]);
      }
    }
    if (s.has_b) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Oct m;
        folded8(vb, at[c], m);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c].p[j] = add2(h[c].p[j], m.p[j]);
      }
    }
    if (s.tok_mod) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Oct m;
        if (a.mscale) {
          smem8_mod(ms + s.scale_at, a.mod_fp32, at[c], m);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[c].p[j] = mul2(h[c].p[j], add2(pair(1.f), m.p[j]));
        }
        if (a.shift) {
          smem8_mod(ms + s.shift_at, a.mod_fp32, at[c], m);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[c].p[j] = add2(h[c].p[j], m.p[j]);
        }
      }
      stage_read(empty);
    }
    const int64_t o = b * a.z_b + t * a.z_n;
    if (a.z_type == kTypeBf16) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (in[c]) put8(static_cast<__nv_bfloat16*>(a.z) + o + at[c], h[c]);
    } else if (a.z_type == kTypeFp32) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (in[c]) put8(static_cast<float*>(a.z) + o + at[c], h[c]);
    } else {
      float m = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        // a copy of the row's last chunk does not change its maximum
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max3_abs_nan(h[c].p[j].x, h[c].p[j].y, m);
      }
      m = row_max_abs(g, m);
      const bool finite = m <= 3.402823466e38f;
      m = finite ? fmaxf(m, kInt8Floor) : m;
      const float inv = __fdiv_rn(127.f, m);
      int8_t* zo = static_cast<int8_t*>(a.z) + o;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // the codes of rows.cuh (code_bits), the products two at a time; a packed sum
          // was contracted with them into one rounding (20 of 20,000 rows of 7,168 had
          // another code; 2 % of the time).  The products and sums with gate, scale and
          // shift above keep their two roundings: the tests hold them to that
          const float2 u = mul2(h[c].p[2 * k], pair(inv)), v = mul2(h[c].p[2 * k + 1], pair(inv));
          const uint32_t lo = __byte_perm(code_of(u.x), code_of(u.y), 0x0040);
          const uint32_t hi = __byte_perm(code_of(v.x), code_of(v.y), 0x0040);
          w[k] = finite ? __byte_perm(lo, hi, 0x5410) : 0u;
        }
        if (in[c]) *reinterpret_cast<uint2*>(zo + at[c]) = make_uint2(w[0], w[1]);
      }
      const float sc = finite ? __fdiv_rn(m, 127.f) : __uint_as_float(0x7fc00000u);
      if (g.tid == 0) a.z_scale[b * a.N + t] = sc;
    }
  }
}

// The ring's shape for these rows, or false where the other kernel runs: rows
// that are short (their loads are in flight enough with one CTA a row), few,
// or too long for two of them beside the vectors in shared memory.
bool ring_shape(const GateNormArgs& a, bool x_fp32, RingShape* s, int* ch, dim3* grid) {
  // scale and shift both once a batch entry (folded) or both once a token (streamed)
  const bool tok_scale = a.mscale && a.scale_n, tok_shift = a.shift && a.shift_n;
  s->tok_mod = tok_scale || tok_shift;
  if (s->tok_mod && ((a.mscale && !tok_scale) || (a.shift && !tok_shift))) return false;
  s->tok_gate = a.gate && a.gate_n;
  s->m_bytes = static_cast<uint32_t>(a.C) * (a.mod_fp32 ? 4 : 2);
  const int per = 148 / a.B > 0 ? 148 / a.B : 1;
  s->x_bytes = static_cast<uint32_t>(a.C) * (x_fp32 ? 4 : 2);
  s->y_bytes = a.y ? static_cast<uint32_t>(a.C) * (a.y_fp32 ? 4 : 2) : 0;
  const int vecs = a.C / 8;
  *ch = vecs <= 32 ? 1 : (vecs <= 64 ? 2 : 4);
  s->threads = ((vecs + *ch - 1) / *ch + 31) / 32 * 32;
  if (s->threads > kRingThreads - 32) return false;
  s->groups = (kRingThreads - 32) / s->threads;
  if (s->threads > 32 && s->groups > kMaxGroups) s->groups = kMaxGroups;
  if (a.N < 4 * per * s->groups || a.B > 65535) return false;
  // short rows: 8 KB a stage and one copy for it, where they lie one after another
  s->rows = 1, s->log_rows = 0;
  s->row_bytes = s->x_bytes + s->y_bytes +
                 (s->tok_gate + (s->tok_mod ? !!a.mscale + !!a.shift : 0)) * s->m_bytes;
  const bool dense = a.x_n == a.C && (!a.y || a.y_n == a.C) && (!s->tok_gate || a.gate_n == a.C) &&
                     (!s->tok_mod || ((!a.mscale || a.scale_n == a.C) && (!a.shift || a.shift_n == a.C)));
  while (dense && s->rows < 16 && s->rows * s->row_bytes < 8192) s->rows *= 2, ++s->log_rows;
  if (s->rows * s->row_bytes < 4096) return false;
  s->has_gain = a.y && ((a.gate && !s->tok_gate) || a.post_weight || a.branch_scale != 1.f);
  s->has_post_bias = a.y && a.post_bias;
  s->has_a = a.z && ((a.mscale && !s->tok_mod) || a.pre_weight);
  s->has_b = a.z && ((a.shift && !s->tok_mod) || a.pre_bias);
  const uint32_t vectors =
      (s->has_gain + s->has_post_bias + s->has_a + s->has_b) * ((a.C + 255) & ~255) * 4u;
  s->off_stage = (vectors + 127) & ~127u;
  const uint32_t fixed = s->groups * static_cast<uint32_t>(sizeof(RowReduce)) + sizeof(RingCtl) + 16;
  const uint32_t stage = s->rows * s->row_bytes;
  s->stage_bytes = stage;
  s->y_at = s->rows * s->x_bytes;
  s->gate_at = s->y_at + s->rows * s->y_bytes;
  s->scale_at = s->gate_at + (s->tok_gate ? s->rows * s->m_bytes : 0);
  s->shift_at = s->scale_at + (s->tok_mod && a.mscale ? s->rows * s->m_bytes : 0);
  if (s->off_stage + fixed + 2 * stage > kRingSmem) return false;
  int stages = static_cast<int>((kRingSmem - s->off_stage - fixed) / stage);
  s->stages = stages < kMaxStages ? stages : kMaxStages;
  // A group waits for its next row's stage by parity: the stage's last filling
  // has to be asked for before the group's own last row was (the kernel's waits),
  // so the stages have to hold as many rows as there are groups.
  if (s->groups > s->stages * s->rows) s->groups = s->stages * s->rows;
  s->off_red = (s->off_stage + s->stages * stage + 15) & ~15u;
  s->off_ctl = s->off_red + s->groups * static_cast<uint32_t>(sizeof(RowReduce));
  s->bytes = s->off_ctl + sizeof(RingCtl);
  *grid = dim3(per, a.B);
  return true;
}

template <class Tx, class Ty, int CH>
cudaError_t launch_ring_ch(const GateNormArgs& a, const RingShape& s, dim3 grid, cudaStream_t st) {
  auto* kernel = gate_norm_ring_kernel<Tx, Ty, CH>;
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_early(kernel, grid, s.groups * s.threads + 32, s.bytes, st, 0, a, s);
}

template <class Tx, class Ty>
cudaError_t launch_ring(const GateNormArgs& a, const RingShape& s, int ch, dim3 grid,
                        cudaStream_t st) {
  if (ch == 1) return launch_ring_ch<Tx, Ty, 1>(a, s, grid, st);
  if (ch == 2) return launch_ring_ch<Tx, Ty, 2>(a, s, grid, st);
  return launch_ring_ch<Tx, Ty, 4>(a, s, grid, st);
}

template <class Tx, int kMode>
cudaError_t launch(const GateNormArgs& a, int ch, int threads, int blocks, cudaStream_t st) {
  auto go = [&](auto k) {
    return launch_early(k, dim3(blocks), threads, 0, st, 0, a);
  };
  if (ch == 1) return go(gate_norm_kernel<Tx, 1, 1024, 1, kMode>);
  if (ch == 2) return threads <= 512 ? go(gate_norm_kernel<Tx, 2, 512, 2, kMode>)
                                     : go(gate_norm_kernel<Tx, 2, 1024, 1, kMode>);
  return go(gate_norm_kernel<Tx, 4, 1024, 1, kMode>);   // rows past 16,384 values: over 512 threads
}

}  // namespace

// Threads and chunks (1, 2 or 4) of a row of n <= 32,768 values: two chunks a
// thread, one for short rows and below `few` rows, where a row's latency counts.
void row_shape(int n, int64_t rows, int few, int* ch, int* threads) {
  const int vecs = (n + 7) / 8;
  int c = rows >= few ? 2 : 1;
  while (c > 1 && (vecs + c - 1) / c < 32) c /= 2;
  while ((vecs + c - 1) / c > 1024) c *= 2;
  *ch = c;
  *threads = ((vecs + c - 1) / c + 31) / 32 * 32;
}

cudaError_t launch_gate_norm(const GateNormArgs& a, bool x_fp32, int mode, cudaStream_t st) {
  RingShape s = {};
  int ch, threads;
  dim3 grid;
  using bf16 = __nv_bfloat16;
  if (mode == kAligned && ring_shape(a, x_fp32, &s, &ch, &grid)) {
    if (x_fp32)
      return a.y_fp32 ? launch_ring<float, float>(a, s, ch, grid, st)
                      : launch_ring<float, bf16>(a, s, ch, grid, st);
    return a.y_fp32 ? launch_ring<bf16, float>(a, s, ch, grid, st)
                    : launch_ring<bf16, bf16>(a, s, ch, grid, st);
  }
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  // few: 512 aligned rows of 7,168 take 11.3 us with two chunks and 17.3 with one; 1,545 odd rows
  // of 1,111, whose chunks cost more instructions, 17.1 and 13.7; 20,000 of 1,001 88 and 105
  const int few = mode == kAligned ? 2 * 148 : 4000;
  row_shape(a.C + (mode == kShifted ? 7 : 0), rows, few, &ch, &threads);
  const int blocks = static_cast<int>(rows < (1 << 30) ? rows : (1 << 30));
  auto go = [&](auto tag) {
    constexpr int kMode = decltype(tag)::value;
    return x_fp32 ? launch<float, kMode>(a, ch, threads, blocks, st)
                  : launch<bf16, kMode>(a, ch, threads, blocks, st);
  };
  if (mode == kAligned) return go(std::integral_constant<int, kAligned>());
  if (mode == kShifted) return go(std::integral_constant<int, kShifted>());
  return go(std::integral_constant<int, kSingles>());
}

}  // namespace bsa
