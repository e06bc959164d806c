// One row of up to 32,768 values spread over a CTA or a group of its warps: loads, stores, the row's
// sums and the int8 codes of a row (gate_norm.cu, quant_int8.cu).
//
// A thread holds CH chunks of 8 values in registers; kMode says which:
//   kAligned  chunk c of thread t is the 8 neighbours at (c threads + t) 8, read
//             and written as 16-byte words (every row starts on one);
//   kShifted  the same moved back by `shift` values, so that the chunks start on
//             16-byte boundaries of rows that do not: rows of an odd length one
//             after another, all operands off by the same amount.  The one or
//             two chunks that a row's ends cut go value by value;
//   kSingles  value j of chunk c sits at (c 8 + j) threads + t: scalar accesses,
//             still contiguous across a warp.
// Everything done to a row is per value or a sum over all of it, so the
// arrangement does not matter to it.
#pragma once

#include "bsa_device.cuh"

namespace bsa {

// Smallest row maximum an int8 scale is taken from: a row of zeros has scale
// 2^-100 / 127 and codes 0, and no scale or its reciprocal leaves fp32's
// normal range.
constexpr float kInt8Floor = 0x1p-100f;

// Per-warp partials of a reduction over the threads of a row.  Uses alternate
// between two slots, so one barrier a reduction is enough: before a slot is
// written again every thread has passed the barrier of the reduction between.
struct RowReduce {
  float4 part[2][32];
  int no[4];           // marks of RowGroup::all (two are used), cleared beforehand
};

// The threads that share a row: a whole CTA, or one of several groups of
// warps in it, each with its own named barrier and partials.
struct RowGroup {
  int tid, threads;    // this thread and the number of threads (whole warps)
  int bar;             // named barrier of the group
  RowReduce* red;
  int turn;            // slot of the next reduction
  int shift;           // values before the row that its first chunk starts at (kShifted)
  __device__ __forceinline__ int warps() const { return threads >> 5; }
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  }
  // True on every thread when it is true on all (one barrier).  A warp that
  // says no leaves a mark before the barrier that all read after it; marks
  // alternate, so a thread that is already at the next one does not disturb.
  // The vote also brings a warp together whose threads came out of a wait one
  // by one, before it arrives at a barrier that counts whole warps.
  __device__ __forceinline__ bool all(bool ok, int& mark) {
    ok = __all_sync(0xffffffffu, ok);
    if (threads == 32) return ok;
    volatile int* no = red->no;
    if (!ok && (tid & 31) == 0) no[mark] = 1;
    sync();
    ok = no[mark] == 0;
    mark ^= 1;
    return ok;
  }
};

enum { kSingles = 0, kAligned = 1, kShifted = 2 };

template <int kMode>
__device__ __forceinline__ int row_index(const RowGroup& g, int c, int j) {
  if (kMode == kSingles) return (c * 8 + j) * g.threads + g.tid;
  return (c * g.threads + g.tid) * 8 + j - (kMode == kShifted ? g.shift : 0);
}
template <int kMode>
__device__ __forceinline__ bool row_in(const RowGroup& g, int c, int j, int n) {
  const int i = row_index<kMode>(g, c, j);
  return kMode == kShifted ? static_cast<unsigned>(i) < static_cast<unsigned>(n) : i < n;
}
// Chunk c lies inside the row and starts on a 16-byte boundary.
template <int kMode>
__device__ __forceinline__ bool row_whole(const RowGroup& g, int c, int n) {
  if (kMode == kSingles) return false;
  const int i = row_index<kMode>(g, c, 0);
  return kMode == kAligned ? i < n : (i >= 0 && i + 8 <= n);
}

__device__ __forceinline__ uint4 ld_row_v4(const void* p) {
  uint4 r;   // not the read-only path: a row may be updated in place
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Values as loaded: a chunk is one (bf16) or two (fp32) 16-byte words.
__device__ __forceinline__ void chunk_words(const __nv_bfloat16* p, float x[8]) {
  bf16x8_to_f32(ld_row_v4(p), x);
}
__device__ __forceinline__ void chunk_words(const float* p, float x[8]) {
  const uint4 a = ld_row_v4(p), b = ld_row_v4(p + 4);
  x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z);
  x[3] = __uint_as_float(a.w), x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y);
  x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
}

// x[c][j] = the row's value, 0 outside it.  A row is read once: it skips L1.
template <int CH, int kMode, class T>
__device__ __forceinline__ void load_row(const RowGroup& g, const T* p, int n, float (&x)[CH][8]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (row_whole<kMode>(g, c, n)) {
      chunk_words(p + row_index<kMode>(g, c, 0), x[c]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[c][j] = kMode != kAligned && row_in<kMode>(g, c, j, n) ? to_f32(p[row_index<kMode>(g, c, j)]) : 0.f;
    }
  }
}

__device__ __forceinline__ void shared_words(const float* p, float v[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void shared_words(const __nv_bfloat16* p, float v[8]) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), v);
}
// 8 neighbours at p, which starts anywhere: from the aligned words around them
// (which lie inside the vector: `room` says so) by a shift that all threads of
// the row share.  8 scalar loads 32 bytes apart across a warp would be 64 passes
// through L1, these are 24.
__device__ __forceinline__ void around8(const float* p, float v[8]) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) >> 2) & 3u;
  const float4* q = reinterpret_cast<const float4*>(p - off);
  const float4 a = *q, b = q[1];
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
  if (off) c = q[2];
  float w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 10; ++j) w[j] = off & 2u ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = off & 1u ? w[j + 1] : w[j];
}
__device__ __forceinline__ bool room(const float* p, int i, int n) {
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p + i) >> 2) & 3u);
  return i >= off && i - off + (off ? 12 : 8) <= n;
}
__device__ __forceinline__ void around8(const __nv_bfloat16* p, float v[8]) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) >> 1) & 7u;
  const uint4* q = reinterpret_cast<const uint4*>(p - off);
  const uint4 a = *q;
  uint4 b = make_uint4(0, 0, 0, 0);
  if (off) b = q[1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = off & 4u ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = off & 2u ? w[j + 1] : w[j];
  uint4 r;
  r.x = off & 1u ? __funnelshift_r(w[0], w[1], 16) : w[0];
  r.y = off & 1u ? __funnelshift_r(w[1], w[2], 16) : w[1];
  r.z = off & 1u ? __funnelshift_r(w[2], w[3], 16) : w[2];
  r.w = off & 1u ? __funnelshift_r(w[3], w[4], 16) : w[3];
  bf16x8_to_f32(r, v);
}
__device__ __forceinline__ bool room(const __nv_bfloat16* p, int i, int n) {
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p + i) >> 1) & 7u);
  return i >= off && i - off + (off ? 16 : 8) <= n;
}

// One chunk of a vector that many rows share (kept in L1); it starts where its
// batch entry does, so that only kAligned chunks start on 16 bytes.
template <int kMode, class T>
__device__ __forceinline__ void load_shared8(const RowGroup& g, const T* p, int n, int c, float v[8]) {
  const int i = row_index<kMode>(g, c, 0);
  if (kMode == kAligned && i < n) {
    shared_words(p + i, v);
  } else if (kMode == kShifted && i >= 0 && room(p, i, n)) {
    around8(p + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = kMode != kAligned && row_in<kMode>(g, c, j, n) ? to_f32(p[row_index<kMode>(g, c, j)]) : 0.f;
  }
}

// One chunk of a row, rounded once to the stored type (to nearest even).
__device__ __forceinline__ void put_chunk(__nv_bfloat16* p, const float v[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void put_chunk(float* p, const float v[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put_value(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_value(float* p, float v) { *p = v; }
template <int kMode, class T>
__device__ __forceinline__ void store8(const RowGroup& g, T* p, int n, int c, const float v[8]) {
  if (row_whole<kMode>(g, c, n)) {
    put_chunk(p + row_index<kMode>(g, c, 0), v);
  } else if (kMode != kAligned) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (row_in<kMode>(g, c, j, n)) put_value(p + row_index<kMode>(g, c, j), v[j]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This lane's share of what every warp of the row left in the current slot
// (warp w's in lane w), after the barrier.
__device__ __forceinline__ float4 row_partials(RowGroup& g, float4 mine) {
  const int lane = g.tid & 31;
  if (lane == 0) g.red->part[g.turn][g.tid >> 5] = mine;
  g.sync();
  const float4 p = lane < g.warps() ? g.red->part[g.turn][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
  g.turn ^= 1;
  return p;
}

// Mean of n values over the row's threads, the quotient rounded once: the
// product with 1 / n, then a step with what it leaves (an overflowed sum stays
// infinite).
__device__ __forceinline__ float row_mean(RowGroup& g, float v, int n) {
  v = warp_sum(v);
  if (g.warps() > 1) v = warp_sum(row_partials(g, make_float4(v, 0.f, 0.f, 0.f)).x);
  const float count = static_cast<float>(n), inv = 1.f / count;
  const float m = v * inv;
  return m <= 3.402823466e38f ? fmaf(fmaf(-m, count, v), inv, m) : m;
}

// Largest value over the row's threads; v >= 0 or NaN, and a NaN anywhere wins (as an
// unsigned word it is above every number).
__device__ __forceinline__ float row_max_abs(RowGroup& g, float v) {
  uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v));
  if (g.warps() > 1)
    m = __reduce_max_sync(0xffffffffu, __float_as_uint(
                              row_partials(g, make_float4(__uint_as_float(m), 0.f, 0.f, 0.f)).x));
  return __uint_as_float(m);
}

// Mean and mean squared deviation of a row of n values from each warp's own
// mean, sum of squares about it and count (exact identity, one barrier).
__device__ __forceinline__ float2 combine_moments(RowGroup& g, float mean, float q, float cnt,
                                                  int n) {
  const float inv = 1.f / n;
  if (g.warps() == 1) return make_float2(mean, q * inv);
  const float4 p = row_partials(g, make_float4(mean, q, cnt, 0.f));
  const float all = warp_sum(p.x * p.z) * inv;
  // nothing from lanes that stand for no values: their distance may square past fp32
  const float d = p.z > 0.f ? p.x - all : 0.f;
  return make_float2(all, warp_sum(fmaf(d * d, p.z, p.y)) * inv);
}

// Mean and mean squared deviation of the row's n values.  Each warp takes the
// mean of its own values and the squares about it, and the warps' results are
// combined exactly (sum of squares + counts x squared distance of the means):
// no difference of large sums, and one barrier.
template <int CH, int kMode>
__device__ __forceinline__ float2 row_moments(RowGroup& g, const float (&x)[CH][8], int n) {
  float s = 0.f, cnt = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s += x[c][j];          // 0 outside the row
    if (kMode == kAligned) {
      cnt += row_whole<kMode>(g, c, n) ? 8.f : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) cnt += row_in<kMode>(g, c, j, n) ? 1.f : 0.f;
    }
  }
  s = warp_sum(s), cnt = warp_sum(cnt);
  const float mean = cnt > 0.f ? s / cnt : 0.f;
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = row_in<kMode>(g, c, j, n);
      const float d = x[c][j] - mean;
      q = in ? fmaf(d, d, q) : q;
    }
  return combine_moments(g, mean, warp_sum(q), cnt, n);
}

// Code of one value, in the low byte: the product is rounded to fp32, and the
// sum with 1.5 2^23 rounds it to a whole number, half to even (|product| <=
// 127.00002), whose two's complement is the sum's low bits.
__device__ __forceinline__ uint32_t code_of(float product) {
  return __float_as_uint(__fadd_rn(product, 12582912.f));
}
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  return code_of(__fmul_rn(x, inv));
}
__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  const uint32_t lo = __byte_perm(code_bits(x[0], inv), code_bits(x[1], inv), 0x0040);
  const uint32_t hi = __byte_perm(code_bits(x[2], inv), code_bits(x[3], inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// int8 codes of a row: scale = amax / 127, code = rint(x * (127 / amax)), both
// factors rounded to fp32, |code| <= 127.  A row that holds a NaN or an
// infinity has a scale that is not finite (NaN) and codes 0: its products are
// NaN.  Stores 8 (or single) codes; returns the scale to every thread.
template <int CH, int kMode>
__device__ __forceinline__ float store_codes(RowGroup& g, const float (&x)[CH][8], int n, int8_t* q) {
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = __float_as_uint(x[c][j]) & 0x7fffffffu;   // 0 outside the row
      m = __uint_as_float(max(__float_as_uint(m), a));
    }
  m = row_max_abs(g, m);
  const bool finite = m <= 3.402823466e38f;
  m = finite ? fmaxf(m, kInt8Floor) : m;
  const float inv = __fdiv_rn(127.f, m);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (kMode == kAligned) {
      uint2 w = make_uint2(0, 0);
      if (finite) w = make_uint2(codes4(x[c], inv), codes4(x[c] + 4, inv));
      if (row_whole<kMode>(g, c, n))
        *reinterpret_cast<uint2*>(q + row_index<kMode>(g, c, 0)) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (row_in<kMode>(g, c, j, n))
          q[row_index<kMode>(g, c, j)] = finite ? static_cast<int8_t>(code_bits(x[c][j], inv)) : 0;
    }
  }
  return finite ? __fdiv_rn(m, 127.f) : __uint_as_float(0x7fc00000u);
}

}  // namespace bsa
