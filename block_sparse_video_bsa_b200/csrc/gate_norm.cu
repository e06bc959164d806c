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
// Two kernels.  gate_norm_ring_kernel for many aligned rows whose vectors are
// shared by the tokens: one CTA per SM keeps the vectors folded together in
// shared memory (three or four loads a row saved), a producer warp streams
// rows through a ring of shared-memory stages with bulk copies, and several
// groups of warps each take the next row, so that the loads in flight do not
// depend on registers and one group's reductions hide behind another's work.
// gate_norm_kernel for the rest: one CTA a row, the row in registers between
// its sums, the vectors from L1 / L2.
#include "bsa_kernels.h"
#include "rows.cuh"

namespace bsa {

namespace {

// ------------------------------------------------------------ one CTA a row

// v = norm(v) * weight + bias, in registers
template <int CH, bool kVec>
__device__ __forceinline__ void norm_row(RowGroup& g, float (&v)[CH][8], int n, int kind, float eps,
                                         const float* weight, const float* bias) {
  if (kind == kNormLayer) {
    const float2 mv = row_moments<CH, kVec>(g, v, n);
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
    const float rs = rsqrtf(row_sum(g, q) / n + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= rs;
  }
  if (weight) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kVec>(g, weight, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] *= w[j];
    }
  }
  if (bias) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      load_shared8<kVec>(g, bias, n, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] += w[j];
    }
  }
}

template <bool kVec>
__device__ __forceinline__ void load_mod8(const RowGroup& g, const void* p, int fp32, int64_t off,
                                          int n, int c, float v[8]) {
  if (fp32)
    load_shared8<kVec>(g, static_cast<const float*>(p) + off, n, c, v);
  else
    load_shared8<kVec>(g, static_cast<const __nv_bfloat16*>(p) + off, n, c, v);
}

template <bool kVec>
__device__ __forceinline__ void store_z8(const RowGroup& g, const GateNormArgs& a, int64_t o, int c,
                                         const float v[8]) {
  if (a.z_type == kTypeBf16)
    store8<kVec>(g, static_cast<__nv_bfloat16*>(a.z) + o, a.C, c, v);
  else if (a.z_type == kTypeFp32)
    store8<kVec>(g, static_cast<float*>(a.z) + o, a.C, c, v);
}

template <class Tx, int CH, int kThreads, int kBlocks, bool kVec>
__global__ void __launch_bounds__(kThreads, kBlocks) gate_norm_kernel(const GateNormArgs a) {
  __shared__ RowReduce red;
  RowGroup g{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 0, &red, 0};
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t b = row / a.N, t = row - b * a.N;
    float h[CH][8];
    load_row<CH, kVec>(g, static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n, a.C, h);
    if (a.y) {
      float y[CH][8];
      const int64_t o = b * a.y_b + t * a.y_n;
      if (a.y_fp32)
        load_row<CH, kVec>(g, static_cast<const float*>(a.y) + o, a.C, y);
      else
        load_row<CH, kVec>(g, static_cast<const __nv_bfloat16*>(a.y) + o, a.C, y);
      norm_row<CH, kVec>(g, y, a.C, a.post, a.eps, a.post_weight, a.post_bias);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (a.gate) {
          float m[8];
          load_mod8<kVec>(g, a.gate, a.mod_fp32, b * a.gate_b + t * a.gate_n, a.C, c, m);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[c][j] *= m[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[c][j] = fmaf(y[c][j], a.branch_scale, h[c][j] * a.residual_scale);
          if (row_index<kVec>(g, c, j) >= a.C) h[c][j] = 0.f;   // a norm reached past the row
        }
        if (a.h) store8<kVec>(g, static_cast<Tx*>(a.h) + b * a.h_b + t * a.h_n, a.C, c, h[c]);
      }
    }
    if (!a.z) continue;
    norm_row<CH, kVec>(g, h, a.C, a.pre, a.eps, a.pre_weight, a.pre_bias);
    const int64_t o = b * a.z_b + t * a.z_n;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.mscale) {
        float m[8];
        load_mod8<kVec>(g, a.mscale, a.mod_fp32, b * a.scale_b + t * a.scale_n, a.C, c, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = fmaf(h[c][j], m[j], h[c][j]);
      }
      if (a.shift) {
        float m[8];
        load_mod8<kVec>(g, a.shift, a.mod_fp32, b * a.shift_b + t * a.shift_n, a.C, c, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += m[j];
      }
      store_z8<kVec>(g, a, o, c, h[c]);
    }
    if (a.z_type == kTypeInt8) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row_index<kVec>(g, c, j) >= a.C) h[c][j] = 0.f;   // a layer norm's mean reached past the row
      const float s = store_codes<CH, kVec>(g, h, a.C, static_cast<int8_t*>(a.z) + o);
      if (g.tid == 0) a.z_scale[row] = s;
    }
  }
}

// ------------------------------------------------------------ rows through a ring

constexpr int kRingThreads = 704;      // 21 warps of rows at most, and the producer warp
constexpr int kMaxGroups = 15;         // named barriers
constexpr int kMaxStages = 16;
constexpr uint32_t kRingSmem = 227 * 1024;

struct RingCtl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort_flag;
};

// What shared memory holds, in floats and bytes.
struct RingShape {
  int threads, groups, stages;   // threads of a group
  int has_gain, has_post_bias;   // gate * post_weight, gate * post_bias
  int has_a, has_b;              // pre_weight (1 + scale), pre_bias (1 + scale) + shift
  uint32_t x_bytes, y_bytes;     // of a row
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

// 8 values as four pairs: the packed fp32 instructions halve the arithmetic,
// which is what bounds this kernel next to HBM.
struct Oct {
  float2 p[4];
};
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
// in[c]: the chunk lies inside the row (the others are copies of its last).
template <int CH, class Get>
__device__ __forceinline__ float2 row_affine(RowGroup& g, int n, int kind, float eps,
                                             const bool (&in)[CH], Get get) {
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
    return make_float2(0.f, rsqrtf(row_sum(g, q) / n + eps));
  }
  // as row_moments (rows.cuh)
  float s = 0.f, cnt = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Oct v;
    get(c, v);
    const float2 t = add2(add2(v.p[0], v.p[1]), add2(v.p[2], v.p[3]));
    s += in[c] ? t.x + t.y : 0.f;
    cnt += in[c] ? 8.f : 0.f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  }
  const float mean = cnt > 0.f ? s / cnt : 0.f;
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
#pragma unroll
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  const float2 mv = combine_moments(g, mean, q, cnt, n);
  const float r = rsqrtf(mv.y + eps);
  return make_float2(-mv.x * r, r);
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
      mbar_init(&ctl->empty[i], s.threads);
    }
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  auto mod = [&](const void* p, int64_t off, int i) {
    return a.mod_fp32 ? __ldg(static_cast<const float*>(p) + off + i)
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[off + i]);
  };
  for (int i = threadIdx.x; i < C; i += blockDim.x) {
    const float gt = a.gate ? mod(a.gate, b * a.gate_b, i) : 1.f;
    const float sc = a.mscale ? 1.f + mod(a.mscale, b * a.scale_b, i) : 1.f;
    const float sh = a.shift ? mod(a.shift, b * a.shift_b, i) : 0.f;
    const int at = folded_at(i);
    if (s.has_gain) gain[at] = a.branch_scale * gt * (a.post_weight ? __ldg(a.post_weight + i) : 1.f);
    if (s.has_post_bias) pbias[at] = a.branch_scale * gt * __ldg(a.post_bias + i);
    if (s.has_a) va[at] = sc * (a.pre_weight ? __ldg(a.pre_weight + i) : 1.f);
    if (s.has_b) vb[at] = fmaf(a.pre_bias ? __ldg(a.pre_bias + i) : 0.f, sc, sh);
  }
  __syncthreads();
  const WaitCtx wc{&ctl->abort_flag, a.dev_status};
  const uint32_t stage_bytes = s.x_bytes + s.y_bytes;
  const int64_t step = gridDim.x;

  if (static_cast<int>(threadIdx.x) >= rows_threads) {
    if (static_cast<int>(threadIdx.x) == rows_threads) {
      int64_t i = 0;
      for (int64_t t = blockIdx.x; t < a.N; t += step, ++i) {
        const int st = static_cast<int>(i % s.stages);
        if (i >= s.stages && !mbar_wait(&ctl->empty[st], ((i / s.stages) - 1) & 1, wc)) break;
        uint8_t* dst = sm + s.off_stage + st * stage_bytes;
        mbar_arrive_expect_tx(&ctl->full[st], stage_bytes);
        bulk_load(dst, static_cast<const Tx*>(a.x) + b * a.x_b + t * a.x_n, s.x_bytes,
                  &ctl->full[st]);
        if (s.y_bytes)
          bulk_load(dst + s.x_bytes, static_cast<const Ty*>(a.y) + b * a.y_b + t * a.y_n, s.y_bytes,
                    &ctl->full[st]);
      }
      // every issued load has landed before the CTA exits
      for (int64_t k = (i > s.stages ? i - s.stages : 0); k < i; ++k)
        mbar_wait(&ctl->full[k % s.stages], (k / s.stages) & 1, wc);
    }
    return;
  }

  const int group = threadIdx.x / s.threads;
  RowGroup g{static_cast<int>(threadIdx.x) - group * s.threads, s.threads, 1 + group,
             reinterpret_cast<RowReduce*>(sm + s.off_red) + group, 0};
  // chunks past the row's end read its last one again and neither count nor store
  int at[CH];
  bool in[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = row_index<true>(g, c, 0);
    in[c] = k < C;
    at[c] = in[c] ? k : C - 8;
  }
  uint32_t st = group % s.stages, round = group / s.stages;
  for (int64_t t = blockIdx.x + group * step; t < a.N; t += s.groups * step) {
    // the whole group goes on or none of it
    if (!g.all(mbar_wait(&ctl->full[st], round & 1, wc))) break;
    const Tx* xs = reinterpret_cast<const Tx*>(sm + s.off_stage + st * stage_bytes);
    const Ty* ys = reinterpret_cast<const Ty*>(sm + s.off_stage + st * stage_bytes + s.x_bytes);
    Oct h[CH];
    if (s.y_bytes) {
      const float2 mr = row_affine<CH>(g, C, a.post, a.eps, in,
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
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Oct x;
        smem8(xs + at[c], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c].p[j] = fma2(x.p[j], pair(a.residual_scale), h[c].p[j]);
      }
      mbar_arrive(&ctl->empty[st]);
      if (a.h) {
        Tx* ho = static_cast<Tx*>(a.h) + b * a.h_b + t * a.h_n;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (in[c]) put8(ho + at[c], h[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) smem8(xs + at[c], h[c]);
      mbar_arrive(&ctl->empty[st]);
    }
    st += s.groups;
    while (st >= static_cast<uint32_t>(s.stages)) st -= s.stages, ++round;
    if (!a.z) continue;
    const float2 mr =
        row_affine<CH>(g, C, a.pre, a.eps, in, [&](int c, Oct& v) { v = h[c]; });
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
      float x[CH][8];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[c][j] = in[c] ? (j & 1 ? h[c].p[j >> 1].y : h[c].p[j >> 1].x) : 0.f;
      const float sc = store_codes<CH, true>(g, x, C, static_cast<int8_t*>(a.z) + o);
      if (g.tid == 0) a.z_scale[b * a.N + t] = sc;
    }
  }
}

// The ring's shape for these rows, or false where the other kernel runs: rows
// that are short (their loads are in flight enough with one CTA a row), few,
// or too long for two of them beside the vectors in shared memory.
bool ring_shape(const GateNormArgs& a, bool x_fp32, RingShape* s, int* ch, dim3* grid) {
  const bool token = (a.gate && a.gate_n) || (a.mscale && a.scale_n) || (a.shift && a.shift_n);
  if (token) return false;
  const int per = 148 / a.B > 0 ? 148 / a.B : 1;
  s->x_bytes = static_cast<uint32_t>(a.C) * (x_fp32 ? 4 : 2);
  s->y_bytes = a.y ? static_cast<uint32_t>(a.C) * (a.y_fp32 ? 4 : 2) : 0;
  if (s->x_bytes + s->y_bytes < 4096) return false;
  const int vecs = a.C / 8;
  *ch = 4;
  s->threads = ((vecs + 3) / 4 + 31) / 32 * 32;
  if (s->threads > kRingThreads - 32) return false;
  s->groups = (kRingThreads - 32) / s->threads;
  if (s->groups > kMaxGroups) s->groups = kMaxGroups;
  // at least four rows a group, or filling the vectors does not pay: 2,000 rows of 1,024 take
  // 12.3 us here and 8.3 us with a CTA a row
  if (a.N < 4 * per * s->groups || a.B > 65535) return false;
  s->has_gain = a.y && (a.gate || a.post_weight || a.branch_scale != 1.f);
  s->has_post_bias = a.y && a.post_bias;
  s->has_a = a.z && (a.mscale || a.pre_weight);
  s->has_b = a.z && (a.shift || a.pre_bias);
  const uint32_t vectors =
      (s->has_gain + s->has_post_bias + s->has_a + s->has_b) * ((a.C + 255) & ~255) * 4u;
  s->off_stage = (vectors + 127) & ~127u;
  const uint32_t fixed = s->groups * static_cast<uint32_t>(sizeof(RowReduce)) + sizeof(RingCtl) + 16;
  const uint32_t stage = s->x_bytes + s->y_bytes;
  if (s->off_stage + fixed + 2 * stage > kRingSmem) return false;
  int stages = static_cast<int>((kRingSmem - s->off_stage - fixed) / stage);
  s->stages = stages < kMaxStages ? stages : kMaxStages;
  s->off_red = (s->off_stage + s->stages * stage + 15) & ~15u;
  s->off_ctl = s->off_red + s->groups * static_cast<uint32_t>(sizeof(RowReduce));
  s->bytes = s->off_ctl + sizeof(RingCtl);
  *grid = dim3(per, a.B);
  return true;
}

template <class Tx, class Ty>
cudaError_t launch_ring(const GateNormArgs& a, const RingShape& s, dim3 grid, cudaStream_t st) {
  auto* kernel = gate_norm_ring_kernel<Tx, Ty, 4>;
  static std::atomic<bool> done[64];
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  });
  if (e != cudaSuccess) return e;
  kernel<<<grid, s.groups * s.threads + 32, s.bytes, st>>>(a, s);
  return cudaGetLastError();
}

template <class Tx, bool kVec>
cudaError_t launch(const GateNormArgs& a, int ch, int threads, int blocks, cudaStream_t st) {
  auto go = [&](auto k) {
    k<<<blocks, threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (ch == 1) return go(gate_norm_kernel<Tx, 1, 1024, 1, kVec>);
  if (ch == 2) return threads <= 512 ? go(gate_norm_kernel<Tx, 2, 512, 2, kVec>)
                                     : go(gate_norm_kernel<Tx, 2, 1024, 1, kVec>);
  return threads <= 512 ? go(gate_norm_kernel<Tx, 4, 512, 1, kVec>)
                        : go(gate_norm_kernel<Tx, 4, 1024, 1, kVec>);
}

}  // namespace

// Threads and chunks (1, 2 or 4) of a row of n <= 32,768 values: two chunks a
// thread, one for short rows and for few rows, where a row's latency counts.
void row_shape(int n, int64_t rows, int* ch, int* threads) {
  const int vecs = (n + 7) / 8;
  int c = rows >= 148 * 2 ? 2 : 1;
  while (c > 1 && (vecs + c - 1) / c < 32) c /= 2;
  while ((vecs + c - 1) / c > 1024) c *= 2;
  *ch = c;
  *threads = ((vecs + c - 1) / c + 31) / 32 * 32;
}

cudaError_t launch_gate_norm(const GateNormArgs& a, bool x_fp32, bool vec, cudaStream_t st) {
  RingShape s = {};
  int ch, threads;
  dim3 grid;
  using bf16 = __nv_bfloat16;
  if (vec && ring_shape(a, x_fp32, &s, &ch, &grid)) {
    if (x_fp32)
      return a.y_fp32 ? launch_ring<float, float>(a, s, grid, st)
                      : launch_ring<float, bf16>(a, s, grid, st);
    return a.y_fp32 ? launch_ring<bf16, float>(a, s, grid, st)
                    : launch_ring<bf16, bf16>(a, s, grid, st);
  }
  const int64_t rows = static_cast<int64_t>(a.B) * a.N;
  row_shape(a.C, rows, &ch, &threads);
  const int blocks = static_cast<int>(rows < (1 << 30) ? rows : (1 << 30));
  if (vec)
    return x_fp32 ? launch<float, true>(a, ch, threads, blocks, st)
                  : launch<bf16, true>(a, ch, threads, blocks, st);
  return x_fp32 ? launch<float, false>(a, ch, threads, blocks, st)
                : launch<bf16, false>(a, ch, threads, blocks, st);
}

}  // namespace bsa
