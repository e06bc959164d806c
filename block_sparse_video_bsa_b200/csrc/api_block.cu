// C ABI of the operators around the attention (declared in include/bsa.h):
// argument checks, tensor maps and launches.  No memory is allocated and no
// state kept.
#include <cmath>
#include <functional>

#include "api_util.h"
#include "bsa.h"
#include "bsa_kernels.h"

namespace {

using bsa::aligned;
using bsa::check_device;
using bsa::cuda_status;

constexpr int kMaxN = 1 << 21;        // tokens a batch entry, as the attention
constexpr int kMaxGrid = 65535;
constexpr int kMaxRow = 32768;        // values of a normed or quantised row; K of the product
constexpr int kMaxSide = 1 << 30;     // rows and columns of the product: tile indices are 32-bit

int type_size(int t) { return t == BSA_DTYPE_BF16 ? 2 : (t == BSA_DTYPE_FP32 ? 4 : 1); }
bool float_type(int t) { return t == BSA_DTYPE_BF16 || t == BSA_DTYPE_FP32; }

// Bytes [lo, hi) that rows of `row` values reach from base.
struct Range {
  uintptr_t lo, hi;
};
Range range_of(const void* base, int size, int64_t row, int64_t n0, int64_t s0, int64_t n1 = 1,
               int64_t s1 = 0, int64_t n2 = 1, int64_t s2 = 0) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
  const unsigned __int128 hi =
      lo + (static_cast<unsigned __int128>(n0 - 1) * s0 + static_cast<unsigned __int128>(n1 - 1) * s1 +
            static_cast<unsigned __int128>(n2 - 1) * s2 + row) * size;
  return Range{lo, hi > UINTPTR_MAX ? UINTPTR_MAX : static_cast<uintptr_t>(hi)};
}
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// A stride in elements; larger ones than 2^40 are no tensor's.
bool stride_ok(int64_t s) { return s >= 0 && s <= (static_cast<int64_t>(1) << 40); }

// Output rows of `row` values must not share elements: each stride of more
// than one entry is at least a row, and sorted strides nest.
bool disjoint(int64_t row, int64_t na, int64_t sa, int64_t nb, int64_t sb, int64_t nc = 1,
              int64_t sc = 0) {
  int64_t n[3] = {na, nb, nc}, s[3] = {sa, sb, sc};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        const int64_t t = s[i], u = n[i];
        s[i] = s[j], n[i] = n[j], s[j] = t, n[j] = u;
      }
  int64_t reach = row;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (s[i] < reach) return false;
    reach = (n[i] - 1) * s[i] + reach;
  }
  return true;
}

// Rows of `row` values of `size` bytes at base, three dimensions of them.
struct Rows {
  const void* base;
  int size;
  int64_t row, n[3], s[3];
  Range range;
  Rows(const void* base, int size, int64_t row, int64_t n0, int64_t s0, int64_t n1, int64_t s1,
       int64_t n2 = 1, int64_t s2 = 0)
      : base(base), size(size), row(row), n{n0, n1, n2}, s{s0, s1, s2},
        range(range_of(base, size, row, n0, s0, n1, s1, n2, s2)) {}
};

// Rows a + i s of wa bytes (i below na in each dimension) and b + j s of wb (j
// below nb), b `at` bytes past a: some share a byte.  Strides in bytes, the
// largest last, each at least what the smaller ones reach, so of every dimension
// only the two steps around `at` can bring them together.
struct Steps {
  int64_t s, na, nb;
};
bool rows_meet(int64_t at, int64_t wa, int64_t wb, const Steps* d, int dims) {
  if (dims == 0) return at < wa && -at < wb;
  const Steps& t = d[dims - 1];
  if (t.na == 1 && t.nb == 1) return rows_meet(at, wa, wb, d, dims - 1);
  const int64_t k0 = at / t.s - (at % t.s < 0);
  for (int64_t k = k0; k <= k0 + 1; ++k)
    if (k < t.na && -k < t.nb && rows_meet(at - k * t.s, wa, wb, d, dims - 1)) return true;
  return false;
}

// No byte belongs to both: their ranges lie apart, or they are rows at the same
// strides that interleave (views of one buffer).
bool apart(const Rows& a, const Rows& b) {
  if (!meet(a.range, b.range)) return true;
  Steps d[3];
  int64_t n[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t sa = a.s[i] * a.size, sb = b.s[i] * b.size;
    const int64_t na = sa ? a.n[i] : 1, nb = sb ? b.n[i] : 1;   // a shared row is one row
    if (na > 1 && nb > 1 && sa != sb) return false;
    d[i] = Steps{na > 1 ? sa : sb, na, nb};
  }
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (d[j].s < d[i].s) {
        const Steps t = d[i];
        d[i] = d[j], d[j] = t;
      }
  for (int i = 0; i < 3; ++i) n[i] = d[i].na > d[i].nb ? d[i].na : d[i].nb;
  const int64_t wa = a.row * a.size, wb = b.row * b.size;
  if (!disjoint(wa > wb ? wa : wb, n[0], d[0].s, n[1], d[1].s, n[2], d[2].s)) return false;
  return !rows_meet(static_cast<int64_t>(b.range.lo - a.range.lo), wa, wb, d, 3);
}

// Each entry checks its arguments and, with `launch`, enqueues its kernel: a
// path of several calls checks all of them before the first launch.

// ------------------------------------------------------------------ rotary

int rotary_entry(const bsa_rotary_params* params, const void* q, const void* k, const void* v,
               const int32_t* positions, const double* freqs, const float* q_weight,
               const float* k_weight, void* Q, void* K, void* V, void* stream, bool launch) {
  if (!params) return BSA_ERR_INVALID;
  bsa_rotary_params own = *params;
  bsa_rotary_params* p = &own;
  if (p->D != 128 || p->B < 1 || p->H < 1 || p->N < 1 || p->N > kMaxN) return BSA_ERR_INVALID;
  if (static_cast<int64_t>(p->B) * 3 > kMaxGrid || p->H > kMaxGrid) return BSA_ERR_INVALID;
  if (p->rotary_dim < 0 || p->rotary_dim > 128 || p->rotary_dim % 2) return BSA_ERR_INVALID;
  if (p->layout != BSA_ROPE_HALF && p->layout != BSA_ROPE_INTERLEAVED) return BSA_ERR_INVALID;
  if (p->axes < 1 || p->axes > 4) return BSA_ERR_INVALID;
  if (!float_type(p->in_dtype) || !float_type(p->out_dtype)) return BSA_ERR_INVALID;
  if (!std::isfinite(p->scale) || !(p->eps >= 0.f) || !std::isfinite(p->eps))
    return BSA_ERR_INVALID;
  bsa::RotaryArgs a = {};
  int pairs = 0;
  for (int i = 0; i < p->axes; ++i) {
    if (p->axis_pairs[i] < 0 || p->axis_pairs[i] > 64) return BSA_ERR_INVALID;
    pairs += p->axis_pairs[i];
    a.axis_end[i] = pairs;
  }
  if (2 * pairs != p->rotary_dim) return BSA_ERR_INVALID;
  if (p->inverse && (q_weight || k_weight)) return BSA_ERR_INVALID;
  // the stride of a single entry is never used
  if (p->B == 1) p->in_b = p->out_b = p->pos_b = 0;
  if (p->H == 1) p->in_h = p->out_h = 0;
  if (p->N == 1) p->in_n = p->out_n = p->pos_n = 0;
  for (int64_t s : {p->in_b, p->in_h, p->in_n, p->out_b, p->out_h, p->out_n, p->pos_b, p->pos_n})
    if (!stride_ok(s)) return BSA_ERR_INVALID;
  if (!disjoint(128, p->B, p->out_b, p->H, p->out_h, p->N, p->out_n)) return BSA_ERR_INVALID;
  const void* in[3] = {q, k, v};
  void* out[3] = {Q, K, V};
  const float* weight[3] = {q_weight, k_weight, nullptr};
  const int si = type_size(p->in_dtype), so = type_size(p->out_dtype);
  const bool same = si == so && p->in_b == p->out_b && p->in_h == p->out_h && p->in_n == p->out_n;
  for (int i = 0; i < 3; ++i) {
    if ((in[i] == nullptr) != (out[i] == nullptr)) return BSA_ERR_INVALID;
    if (!in[i]) {
      if (weight[i]) return BSA_ERR_INVALID;
      continue;
    }
    a.in[a.ntens] = in[i];
    a.out[a.ntens] = out[i];
    a.weight[a.ntens] = weight[i];
    a.turn[a.ntens] = i < 2;
    ++a.ntens;
  }
  if (a.ntens == 0) return BSA_ERR_INVALID;
  if (p->rotary_dim > 0 && (q || k) && (!positions || !freqs)) return BSA_ERR_INVALID;
  // Outputs: on their own input exactly, or apart from every input and output.
  auto ins = [&](int i) {
    return Rows(a.in[i], si, 128, p->B, p->in_b, p->H, p->in_h, p->N, p->in_n);
  };
  auto outs = [&](int i) {
    return Rows(a.out[i], so, 128, p->B, p->out_b, p->H, p->out_h, p->N, p->out_n);
  };
  const Rows rin[3] = {ins(0), ins(1), ins(2)}, rout[3] = {outs(0), outs(1), outs(2)};
  for (int i = 0; i < a.ntens; ++i)
    for (int j = 0; j < a.ntens; ++j) {
      const bool in_place = i == j && a.out[i] == a.in[i] && same;
      if (!in_place && !apart(rout[i], rin[j])) return BSA_ERR_INVALID;
      if (j > i && !apart(rout[i], rout[j])) return BSA_ERR_INVALID;
    }
  for (int i = 0; i < a.ntens; ++i)
    if (!aligned(a.in[i], 16) || !aligned(a.out[i], 16) ||
        (a.weight[i] && !aligned(a.weight[i], 16)))
      return BSA_ERR_ALIGN;
  for (int64_t s : {p->in_b, p->in_h, p->in_n})
    if (s * si % 16) return BSA_ERR_ALIGN;
  for (int64_t s : {p->out_b, p->out_h, p->out_n})
    if (s * so % 16) return BSA_ERR_ALIGN;
  if ((positions && !aligned(positions, 4)) || (freqs && !aligned(freqs, 8))) return BSA_ERR_ALIGN;
  if (!launch) return BSA_OK;
  int rc = check_device();
  if (rc) return rc;
  a.B = p->B, a.H = p->H, a.N = p->N, a.r = p->rotary_dim;
  a.interleaved = p->layout == BSA_ROPE_INTERLEAVED;
  a.scale = p->scale;
  a.sin_scale = p->inverse ? -p->scale : p->scale;
  a.eps = p->eps;
  a.in_b = p->in_b, a.in_h = p->in_h, a.in_n = p->in_n;
  a.out_b = p->out_b, a.out_h = p->out_h, a.out_n = p->out_n;
  a.pos_b = p->pos_b, a.pos_n = p->pos_n;
  a.positions = positions;
  a.freqs = freqs;
  return cuda_status(bsa::launch_rotary(a, p->in_dtype == BSA_DTYPE_FP32,
                                        p->out_dtype == BSA_DTYPE_FP32,
                                        static_cast<cudaStream_t>(stream)));
}

// q, k and v with parameters of their own: every check before the first launch,
// then one launch for each set of tensors that lie alike.
int rotary_each_entry(const bsa_rotary_params* p, const void* const (&in)[3],
                      const int32_t* positions, const double* freqs, const float* const (&weight)[3],
                      void* const (&out)[3], void* stream) {
  if (!p) return BSA_ERR_INVALID;
  int first = -1, set[3];
  auto rows = [&](int i, bool input) {
    const bsa_rotary_params& r = p[i];
    const int size = type_size(input ? r.in_dtype : r.out_dtype);
    if (input) return Rows(in[i], size, 128, r.B, r.in_b, r.H, r.in_h, r.N, r.in_n);
    return Rows(out[i], size, 128, r.B, r.out_b, r.H, r.out_h, r.N, r.out_n);
  };
  auto alike = [](const Rows& a, const Rows& b) {
    bool same = a.size == b.size;
    for (int d = 0; d < 3; ++d)
      same = same && a.n[d] == b.n[d] && (a.n[d] == 1 || a.s[d] == b.s[d]);
    return same;
  };
  // the tensors `from` and on of set `s` (all where s is negative), as bsa_rotary takes them
  auto run = [&](int from, int s, bool launch) {
    const void* x[3] = {};
    void* y[3] = {};
    const float* w[3] = {};
    for (int i = from; i < (s < 0 ? from + 1 : 3); ++i)
      if (s < 0 || (in[i] && set[i] == s)) x[i] = in[i], y[i] = out[i], w[i] = weight[i];
    return rotary_entry(p + from, x[0], x[1], x[2], positions, freqs, w[0], w[1], y[0], y[1], y[2],
                        stream, launch);
  };
  for (int i = 0; i < 3; ++i) {
    if (!in[i] && !out[i] && !weight[i]) continue;
    const int rc = run(i, -1, false);
    if (rc) return rc;
    if (first < 0) first = i;
    const bsa_rotary_params &a = p[first], &b = p[i];
    bool one = a.B == b.B && a.N == b.N && a.rotary_dim == b.rotary_dim && a.layout == b.layout &&
               a.axes == b.axes && !a.inverse == !b.inverse && a.scale == b.scale &&
               a.eps == b.eps && (a.B == 1 || a.pos_b == b.pos_b) && (a.N == 1 || a.pos_n == b.pos_n);
    for (int d = 0; one && d < a.axes; ++d) one = a.axis_pairs[d] == b.axis_pairs[d];
    if (!one) return BSA_ERR_INVALID;
    set[i] = i;
    for (int j = first; j < i; ++j)
      if (in[j] && set[i] == i && alike(rows(i, true), rows(j, true)) &&
          alike(rows(i, false), rows(j, false)))
        set[i] = set[j];
  }
  if (first < 0) return BSA_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j) {
      if (!in[i] || !in[j]) continue;
      const Rows o = rows(i, false), x = rows(j, true);
      const bool in_place = i == j && o.base == x.base && alike(o, x);
      if (!in_place && !apart(o, x)) return BSA_ERR_INVALID;
      if (j > i && !apart(o, rows(j, false))) return BSA_ERR_INVALID;
    }
  for (int i = first; i < 3; ++i) {
    if (!in[i] || set[i] != i) continue;
    const int rc = run(i, i, true);
    if (rc) return rc;
  }
  return BSA_OK;
}

// ------------------------------------------------------------------ gate norm

int gate_norm_entry(const bsa_gate_norm_params* params, const bsa_gate_norm_inputs* in, void* h, void* z,
                  float* z_scale, void* stream, bool launch) {
  if (!params || !in) return BSA_ERR_INVALID;
  bsa_gate_norm_params own = *params;
  bsa_gate_norm_params* p = &own;
  if (p->B < 1 || p->N < 1 || p->C < 1 || p->C > kMaxRow) return BSA_ERR_INVALID;
  for (int kind : {p->pre, p->post})
    if (kind < BSA_NORM_NONE || kind > BSA_NORM_LAYER) return BSA_ERR_INVALID;
  if (!float_type(p->x_dtype) || !float_type(p->y_dtype) || !float_type(p->mod_dtype))
    return BSA_ERR_INVALID;
  if (!float_type(p->z_dtype) && p->z_dtype != BSA_DTYPE_INT8) return BSA_ERR_INVALID;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->residual_scale) ||
      !std::isfinite(p->branch_scale))
    return BSA_ERR_INVALID;
  if (!in->x || (!h && !z)) return BSA_ERR_INVALID;
  if (!in->y && (h || in->gate)) return BSA_ERR_INVALID;
  if (!z && (in->scale || in->shift || in->pre_weight || in->pre_bias)) return BSA_ERR_INVALID;
  if ((z && p->z_dtype == BSA_DTYPE_INT8) != (z_scale != nullptr)) return BSA_ERR_INVALID;
  // the stride of a single entry is never used
  if (p->B == 1)
    p->x_b = p->y_b = p->h_b = p->z_b = p->gate_b = p->scale_b = p->shift_b = 0;
  if (p->N == 1)
    p->x_n = p->y_n = p->h_n = p->z_n = p->gate_n = p->scale_n = p->shift_n = 0;
  for (int64_t s : {p->x_b, p->x_n, p->y_b, p->y_n, p->h_b, p->h_n, p->z_b, p->z_n, p->gate_b,
                    p->gate_n, p->scale_b, p->scale_n, p->shift_b, p->shift_n})
    if (!stride_ok(s)) return BSA_ERR_INVALID;
  const int sx = type_size(p->x_dtype), sy = type_size(p->y_dtype), sm = type_size(p->mod_dtype),
            sz = type_size(p->z_dtype);
  if (h && !disjoint(p->C, p->B, p->h_b, p->N, p->h_n)) return BSA_ERR_INVALID;
  if (z && !disjoint(p->C, p->B, p->z_b, p->N, p->z_n)) return BSA_ERR_INVALID;
  // h may be x itself (the residual updated in place); any other overlap of an
  // output is refused, with the vectors too: one a token is as large as the rows,
  // and is read after other rows were written.
  auto rows = [&](const void* base, int size, int64_t sb, int64_t sn) {
    return Rows(base, size, p->C, p->B, sb, p->N, sn);
  };
  const Rows x = rows(in->x, sx, p->x_b, p->x_n), y = rows(in->y, sy, p->y_b, p->y_n);
  const Rows ho = rows(h, sx, p->h_b, p->h_n), zo = rows(z, sz, p->z_b, p->z_n);
  const Rows vectors[7] = {rows(in->gate, sm, p->gate_b, p->gate_n),
                           rows(in->scale, sm, p->scale_b, p->scale_n),
                           rows(in->shift, sm, p->shift_b, p->shift_n),
                           rows(in->post_weight, 4, 0, 0), rows(in->post_bias, 4, 0, 0),
                           rows(in->pre_weight, 4, 0, 0), rows(in->pre_bias, 4, 0, 0)};
  const bool in_place = h == in->x && p->h_b == p->x_b && p->h_n == p->x_n;
  if (h && z && !apart(ho, zo)) return BSA_ERR_INVALID;
  for (const Rows& o : {std::cref(ho), std::cref(zo)}) {
    if (!o.base) continue;
    if (!(o.base == h && in_place) && !apart(o, x)) return BSA_ERR_INVALID;
    if (in->y && !apart(o, y)) return BSA_ERR_INVALID;
    for (const Rows& v : vectors)
      if (v.base && !apart(o, v)) return BSA_ERR_INVALID;
  }
  if (!aligned(in->x, sx) || (in->y && !aligned(in->y, sy)) || (h && !aligned(h, sx)) ||
      (z && !aligned(z, sz)) || (z_scale && !aligned(z_scale, 4)))
    return BSA_ERR_ALIGN;
  for (const void* m : {in->gate, in->scale, in->shift})
    if (m && !aligned(m, sm)) return BSA_ERR_ALIGN;
  for (const float* w : {in->post_weight, in->post_bias, in->pre_weight, in->pre_bias})
    if (w && !aligned(w, 4)) return BSA_ERR_ALIGN;
  if (!launch) return BSA_OK;
  int rc = check_device();
  if (rc) return rc;
  bsa::GateNormArgs a = {};
  a.x = in->x, a.y = in->y, a.gate = in->gate, a.mscale = in->scale, a.shift = in->shift;
  a.post_weight = in->y ? in->post_weight : nullptr;
  a.post_bias = in->y ? in->post_bias : nullptr;
  a.pre_weight = in->pre_weight, a.pre_bias = in->pre_bias;
  a.h = h, a.z = z, a.z_scale = z_scale;
  a.B = p->B, a.N = p->N, a.C = p->C, a.pre = p->pre, a.post = p->post;
  a.y_fp32 = p->y_dtype == BSA_DTYPE_FP32, a.mod_fp32 = p->mod_dtype == BSA_DTYPE_FP32;
  a.z_type = p->z_dtype;
  a.dev_status = p->dev_status;
  a.eps = p->eps, a.residual_scale = p->residual_scale, a.branch_scale = p->branch_scale;
  a.x_b = p->x_b, a.x_n = p->x_n, a.y_b = p->y_b, a.y_n = p->y_n, a.h_b = p->h_b, a.h_n = p->h_n;
  a.z_b = p->z_b, a.z_n = p->z_n, a.gate_b = p->gate_b, a.gate_n = p->gate_n;
  a.scale_b = p->scale_b, a.scale_n = p->scale_n, a.shift_b = p->shift_b, a.shift_n = p->shift_n;
  // How the rows lie: aligned (1) where every row of every operand starts on
  // 16 bytes (8 codes: 8 bytes); shifted (2) where the rows of x, y, h, z and of
  // per-token vectors are all off by the same number of values; else singles (0).
  bool vec = p->C % 8 == 0, same = true;
  auto row = [&](const void* base, int size, int64_t sb, int64_t sn) {
    if (!base) return;
    const bool start = aligned(base, 8 * size < 16 ? 8 * size : 16);
    vec = vec && start && sb % 8 == 0 && sn % 8 == 0;
    same = same && start && (sb - p->x_b) % 8 == 0 && (sn - p->x_n) % 8 == 0;
  };
  auto vector = [&](const void* base, int size, int64_t sb, int64_t sn) {
    if (base && sn != 0) return row(base, size, sb, sn);
    if (base) vec = vec && aligned(base, 16) && sb % 8 == 0;
  };
  row(in->x, sx, p->x_b, p->x_n);
  row(in->y, sy, p->y_b, p->y_n);
  row(h, sx, p->h_b, p->h_n);
  if (p->z_dtype != BSA_DTYPE_INT8)
    row(z, sz, p->z_b, p->z_n);
  else if (z)                       // codes are written one by one where they are not aligned
    vec = vec && aligned(z, 8) && p->z_b % 8 == 0 && p->z_n % 8 == 0;
  vector(in->gate, sm, p->gate_b, p->gate_n);
  vector(in->scale, sm, p->scale_b, p->scale_n);
  vector(in->shift, sm, p->shift_b, p->shift_n);
  for (const float* w : {in->post_weight, in->post_bias, in->pre_weight, in->pre_bias})
    vector(w, 4, 0, 0);
  const int mode = vec ? 1 : (same && p->C + 7 <= kMaxRow ? 2 : 0);   // the shift takes room for 7
  return cuda_status(bsa::launch_gate_norm(a, p->x_dtype == BSA_DTYPE_FP32, mode,
                                           static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ int8

int quantize_int8_entry(const bsa_quantize_int8_params* params, const void* x, int8_t* codes, float* scale,
                      void* stream, bool launch) {
  if (!params) return BSA_ERR_INVALID;
  bsa_quantize_int8_params own = *params;
  bsa_quantize_int8_params* p = &own;
  if (p->B < 1 || p->N < 1 || p->S < 1 || p->L < 1) return BSA_ERR_INVALID;
  if (static_cast<int64_t>(p->S) * p->L > kMaxRow) return BSA_ERR_INVALID;
  if (static_cast<int64_t>(p->B) * p->N > INT32_MAX) return BSA_ERR_INVALID;
  if (!float_type(p->x_dtype)) return BSA_ERR_INVALID;
  if (!x || !codes || !scale) return BSA_ERR_INVALID;
  // the stride of a single entry is never used
  if (p->B == 1) p->x_b = 0;
  if (p->N == 1) p->x_n = 0;
  if (p->S == 1) p->x_s = 0;
  if (p->B == 1 && p->N == 1) p->ld = static_cast<int64_t>(p->S) * p->L;
  for (int64_t s : {p->x_b, p->x_n, p->x_s, p->ld})
    if (!stride_ok(s)) return BSA_ERR_INVALID;
  const int64_t K = static_cast<int64_t>(p->S) * p->L;
  const int64_t rows = static_cast<int64_t>(p->B) * p->N;
  if (p->ld < K) return BSA_ERR_INVALID;
  const int sx = type_size(p->x_dtype);
  if (meet(range_of(x, sx, p->L, p->B, p->x_b, p->N, p->x_n, p->S, p->x_s),
           range_of(codes, 1, K, rows, p->ld)))
    return BSA_ERR_INVALID;
  if (!aligned(x, sx) || !aligned(scale, 4)) return BSA_ERR_ALIGN;
  if (!launch) return BSA_OK;
  int rc = check_device();
  if (rc) return rc;
  bsa::QuantInt8Args a = {};
  a.x = x, a.q = codes, a.scale = scale;
  a.B = p->B, a.N = p->N, a.S = p->S, a.L = p->L;
  a.x_b = p->x_b, a.x_n = p->x_n, a.x_s = p->x_s, a.q_ld = p->ld;
  const bool vec = p->L % 8 == 0 && aligned(x, 16) && aligned(codes, 8) &&
                   p->x_b % 8 == 0 && p->x_n % 8 == 0 && p->x_s % 8 == 0 &&
                   (rows == 1 || p->ld % 8 == 0);
  return cuda_status(bsa::launch_quant_int8(a, p->x_dtype == BSA_DTYPE_FP32, vec,
                                            static_cast<cudaStream_t>(stream)));
}

int linear_int8_entry(const bsa_linear_int8_params* params, const int8_t* a, const float* a_scale,
                    const int8_t* w, const float* w_scale, const float* bias, void* out,
                    void* stream, bool launch) {
  if (!params) return BSA_ERR_INVALID;
  bsa_linear_int8_params own = *params;
  bsa_linear_int8_params* p = &own;
  if (p->M < 1 || p->N < 1 || p->K < 1 || p->K > kMaxRow) return BSA_ERR_INVALID;
  if (p->M > kMaxSide || p->N > kMaxSide) return BSA_ERR_INVALID;
  if (!float_type(p->out_dtype)) return BSA_ERR_INVALID;
  if (!a || !a_scale || !w || !w_scale || !out) return BSA_ERR_INVALID;
  // the stride of a single row is never used
  if (p->M == 1) p->lda = (p->K + 15) / 16 * 16, p->ldo = p->N;
  if (p->N == 1) p->ldw = (p->K + 15) / 16 * 16;
  for (int64_t s : {p->lda, p->ldw, p->ldo})
    if (!stride_ok(s)) return BSA_ERR_INVALID;
  if (p->lda < p->K || p->ldw < p->K || p->ldo < p->N) return BSA_ERR_INVALID;
  const int so = type_size(p->out_dtype);
  const Range ro = range_of(out, so, p->N, p->M, p->ldo);
  if (meet(ro, range_of(a, 1, p->K, p->M, p->lda)) || meet(ro, range_of(w, 1, p->K, p->N, p->ldw)))
    return BSA_ERR_INVALID;
  if (!aligned(a, 16) || !aligned(w, 16) || p->lda % 16 || p->ldw % 16 || !aligned(out, so) ||
      !aligned(a_scale, 4) || !aligned(w_scale, 4) || (bias && !aligned(bias, 4)))
    return BSA_ERR_ALIGN;
  if (!launch) return BSA_OK;
  int rc = check_device();
  if (rc) return rc;
  bsa::EncodeTiledFn enc = bsa::encode_fn();
  if (!enc) return BSA_ERR_UNSUPPORTED;
  // rows of K bytes, `box` of them 128 bytes wide; what lies past K or the
  // last row reads as zero
  auto map = [&](CUtensorMap* m, const int8_t* base, int rows, int64_t ld, int box) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p->K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t b[2] = {128, static_cast<cuuint32_t>(box)}, one[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, b,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  int box_a, box_w;
  bsa::linear_int8_boxes(p->M, p->N, &box_a, &box_w);
  CUtensorMap ma, mw;
  if (!map(&ma, a, p->M, p->lda, box_a) || !map(&mw, w, p->N, p->ldw, box_w))
    return BSA_ERR_UNSUPPORTED;
  bsa::LinearInt8Args l = {};
  l.M = p->M, l.N = p->N, l.K = p->K;
  l.a_scale = a_scale, l.w_scale = w_scale, l.bias = bias;
  l.out = out, l.ldo = p->ldo, l.out_fp32 = p->out_dtype == BSA_DTYPE_FP32;
  l.dev_status = p->dev_status;
  return cuda_status(bsa::launch_linear_int8(l, ma, mw, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ block path

// Intermediates of the block path carved from one buffer (each piece 256-byte
// aligned).  What follows the attention takes the place of the projection.
struct BlockWs {
  int8_t* z8;
  float* zs;
  uint8_t* qkv;                 // bf16 [B, N, 3, H, 128]
  uint8_t *Q, *K, *V;
  uint8_t* O;                   // over qkv
  int8_t* o8;
  float* os;
  uint8_t* y;
  uint8_t* attn;
};

size_t block_carve(const bsa_params* p, int C, uint8_t* base, BlockWs* w) {
  const size_t rows = static_cast<size_t>(p->B) * p->N, hd = static_cast<size_t>(p->H) * 128;
  const size_t ldc = (static_cast<size_t>(C) + 15) / 16 * 16;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base ? base + off : nullptr;
    off += bsa::round256(bytes);
    return q;
  };
  BlockWs o = {};
  o.z8 = reinterpret_cast<int8_t*>(take(rows * ldc));
  o.zs = reinterpret_cast<float*>(take(rows * 4));
  o.Q = take(rows * hd * 2);
  o.K = take(rows * hd * 2);
  o.V = take(rows * hd * 2);
  o.attn = take(bsa_workspace_bytes(p));
  const size_t mark = off;
  o.qkv = take(rows * 3 * hd * 2);
  const size_t first = off;
  off = mark;
  o.O = take(rows * hd * 2);
  o.o8 = reinterpret_cast<int8_t*>(take(rows * hd));
  o.os = reinterpret_cast<float*>(take(rows * 4));
  o.y = take(rows * C * 2);
  if (off < first) off = first;
  if (w) *w = o;
  return off;
}

// The calls of the path on one workspace; with launch = false only their checks.
int block_run(const bsa_params* p, const bsa_block_params* bp, const bsa_block_weights* bw,
              const void* x, void* out, const BlockWs& w, void* stream, bool launch) {
  const int B = p->B, N = p->N, H = p->H, C = bp->C;
  const int64_t hd = static_cast<int64_t>(H) * 128, ldc = (C + 15) / 16 * 16;
  bsa_gate_norm_params g = {};
  g.B = B, g.N = N, g.C = C, g.pre = bp->pre, g.post = bp->post;
  g.x_dtype = bp->x_dtype, g.mod_dtype = bp->mod_dtype;
  g.y_dtype = BSA_DTYPE_BF16, g.z_dtype = BSA_DTYPE_INT8;
  g.eps = bp->eps, g.residual_scale = bp->residual_scale, g.branch_scale = bp->branch_scale;
  g.x_b = g.y_b = g.h_b = static_cast<int64_t>(N) * C;
  g.x_n = g.y_n = g.h_n = C;
  g.z_b = N * ldc, g.z_n = ldc;
  g.gate_b = bp->gate_b, g.gate_n = bp->gate_n, g.scale_b = bp->scale_b, g.scale_n = bp->scale_n;
  g.shift_b = bp->shift_b, g.shift_n = bp->shift_n;
  g.dev_status = p->dev_status;
  bsa_gate_norm_inputs in = {};
  in.x = x, in.scale = bw->scale, in.shift = bw->shift;
  in.pre_weight = bw->pre_weight, in.pre_bias = bw->pre_bias;
  int rc = gate_norm_entry(&g, &in, nullptr, w.z8, w.zs, stream, launch);
  if (rc) return rc;

  bsa_linear_int8_params l = {};
  l.M = B * N, l.N = static_cast<int>(3 * hd), l.K = C, l.out_dtype = BSA_DTYPE_BF16;
  l.lda = ldc, l.ldw = bp->ld_qkv, l.ldo = 3 * hd, l.dev_status = p->dev_status;
  if ((rc = linear_int8_entry(&l, w.z8, w.zs, bw->w_qkv, bw->s_qkv, bw->b_qkv, w.qkv, stream,
                              launch)))
    return rc;

  bsa_rotary_params r = {};
  r.B = B, r.H = H, r.N = N, r.D = p->D;
  r.rotary_dim = bp->rotary_dim, r.layout = bp->layout, r.axes = bp->axes;
  for (int i = 0; i < 4; ++i) r.axis_pairs[i] = bp->axis_pairs[i];
  r.in_dtype = r.out_dtype = BSA_DTYPE_BF16;
  r.scale = bp->rope_scale, r.eps = bp->qk_eps;
  r.in_b = N * 3 * hd, r.in_n = 3 * hd, r.in_h = 128;
  r.out_b = N * hd, r.out_h = static_cast<int64_t>(N) * 128, r.out_n = 128;
  r.pos_b = bp->pos_b, r.pos_n = bp->pos_n;
  if ((rc = rotary_entry(&r, w.qkv, w.qkv + hd * 2, w.qkv + 2 * hd * 2, bw->positions, bw->freqs,
                         bw->q_weight, bw->k_weight, w.Q, w.K, w.V, stream, launch)))
    return rc;

  if (launch && (rc = bsa_forward(p, w.Q, w.K, w.V, w.O, nullptr, w.attn, bsa_workspace_bytes(p),
                                  stream)))
    return rc;

  bsa_quantize_int8_params q = {};
  q.B = B, q.N = N, q.S = H, q.L = 128, q.x_dtype = BSA_DTYPE_BF16;
  q.x_b = N * hd, q.x_n = 128, q.x_s = static_cast<int64_t>(N) * 128, q.ld = hd;
  if ((rc = quantize_int8_entry(&q, w.O, w.o8, w.os, stream, launch))) return rc;

  l.N = C, l.K = static_cast<int>(hd), l.lda = hd, l.ldw = bp->ld_out, l.ldo = C;
  if ((rc = linear_int8_entry(&l, w.o8, w.os, bw->w_out, bw->s_out, bw->b_out, w.y, stream, launch)))
    return rc;

  in = {};
  in.x = x, in.y = w.y, in.gate = bw->gate;
  in.post_weight = bw->post_weight, in.post_bias = bw->post_bias;
  g.z_dtype = BSA_DTYPE_BF16;
  return gate_norm_entry(&g, &in, out, nullptr, nullptr, stream, launch);
}

bool block_valid(const bsa_params* p, const bsa_block_params* bp) {
  return p && bp && bsa_workspace_bytes(p) != 0 && bp->C >= 1 && bp->C <= kMaxRow &&
         p->H <= kMaxRow / 128 && static_cast<int64_t>(p->B) * p->N <= INT32_MAX;
}

}  // namespace

extern "C" {

int bsa_rotary_freqs(int32_t pairs, double base, int32_t scaling, double factor,
                     double trained_length, double fast_turns, double slow_turns, double* freqs,
                     float* scale) {
  if (pairs < 0 || pairs > 64 || (pairs > 0 && !freqs) || !scale) return BSA_ERR_INVALID;
  if (!(base > 1.0) || !std::isfinite(base)) return BSA_ERR_INVALID;
  if (scaling < BSA_ROPE_PLAIN || scaling > BSA_ROPE_BY_PARTS) return BSA_ERR_INVALID;
  const bool by_parts = scaling == BSA_ROPE_YARN || scaling == BSA_ROPE_BY_PARTS;
  if (scaling != BSA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return BSA_ERR_INVALID;
  if (by_parts && (!(trained_length >= 1.0) || !std::isfinite(trained_length) ||
                   !(fast_turns > slow_turns) || !(slow_turns >= 0.0) ||
                   !std::isfinite(fast_turns)))
    return BSA_ERR_INVALID;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == BSA_ROPE_NTK && pairs > 1)
    base *= std::pow(factor, static_cast<double>(pairs) / (pairs - 1));
  for (int i = 0; i < pairs; ++i) {
    double f = std::pow(base, -static_cast<double>(i) / pairs);
    if (scaling == BSA_ROPE_LINEAR) f /= factor;
    if (by_parts) {
      // share of the pair's own frequency: 1 from fast_turns over the trained
      // length on, 0 up to slow_turns
      const double turns = trained_length * f / two_pi;
      double keep = (turns - slow_turns) / (fast_turns - slow_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    freqs[i] = f;
  }
  *scale = scaling == BSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return BSA_OK;
}

int bsa_rotary(const bsa_rotary_params* params, const void* q, const void* k, const void* v,
               const int32_t* positions, const double* freqs, const float* q_weight,
               const float* k_weight, void* Q, void* K, void* V, void* stream) {
  return rotary_entry(params, q, k, v, positions, freqs, q_weight, k_weight, Q, K, V, stream, true);
}

int bsa_rotary_each(const bsa_rotary_params* params, const void* q, const void* k, const void* v,
                    const int32_t* positions, const double* freqs, const float* q_weight,
                    const float* k_weight, void* Q, void* K, void* V, void* stream) {
  const void* const in[3] = {q, k, v};
  void* const out[3] = {Q, K, V};
  const float* const weight[3] = {q_weight, k_weight, nullptr};
  return rotary_each_entry(params, in, positions, freqs, weight, out, stream);
}

int bsa_gate_norm(const bsa_gate_norm_params* params, const bsa_gate_norm_inputs* in, void* h, void* z,
                  float* z_scale, void* stream) {
  return gate_norm_entry(params, in, h, z, z_scale, stream, true);
}

int bsa_quantize_int8(const bsa_quantize_int8_params* params, const void* x, int8_t* codes, float* scale,
                      void* stream) {
  return quantize_int8_entry(params, x, codes, scale, stream, true);
}

int bsa_linear_int8(const bsa_linear_int8_params* params, const int8_t* a, const float* a_scale,
                    const int8_t* w, const float* w_scale, const float* bias, void* out,
                    void* stream) {
  return linear_int8_entry(params, a, a_scale, w, w_scale, bias, out, stream, true);
}

size_t bsa_forward_block_workspace_bytes(const bsa_params* p, const bsa_block_params* bp) {
  return block_valid(p, bp) ? block_carve(p, bp->C, nullptr, nullptr) : 0;
}

int bsa_forward_block(const bsa_params* p, const bsa_block_params* bp, const bsa_block_weights* w,
                      const void* x, void* out, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!block_valid(p, bp) || !w || !x || !out || !workspace) return BSA_ERR_INVALID;
  if (workspace_bytes < block_carve(p, bp->C, nullptr, nullptr)) return BSA_ERR_INVALID;
  if (!aligned(workspace, 256)) return BSA_ERR_ALIGN;
  // the workspace lies apart from the rows that are read and written
  const int64_t rows = static_cast<int64_t>(p->B) * p->N;
  if (!float_type(bp->x_dtype)) return BSA_ERR_INVALID;
  const int sx = type_size(bp->x_dtype);
  const Range ws{reinterpret_cast<uintptr_t>(workspace),
                 reinterpret_cast<uintptr_t>(workspace) + block_carve(p, bp->C, nullptr, nullptr)};
  if (meet(ws, range_of(x, sx, bp->C, rows, bp->C)) || meet(ws, range_of(out, sx, bp->C, rows, bp->C)))
    return BSA_ERR_INVALID;
  // and it and the result apart from the weights and vectors
  const int64_t hd = static_cast<int64_t>(p->H) * 128, C = bp->C;
  const int sm = type_size(bp->mod_dtype);
  const struct {
    const void* base;
    int size;
    int64_t row, n0, s0, n1, s1;
  } read[] = {{w->w_qkv, 1, C, 3 * hd, bp->ld_qkv, 1, 0},
              {w->w_out, 1, hd, C, bp->ld_out, 1, 0},
              {w->gate, sm, C, p->B, bp->gate_b, p->N, bp->gate_n},
              {w->scale, sm, C, p->B, bp->scale_b, p->N, bp->scale_n},
              {w->shift, sm, C, p->B, bp->shift_b, p->N, bp->shift_n},
              {w->positions, 4, bp->axes, p->B, bp->pos_b, p->N, bp->pos_n},
              {w->s_qkv, 4, 3 * hd, 1, 0, 1, 0},
              {w->b_qkv, 4, 3 * hd, 1, 0, 1, 0},
              {w->s_out, 4, C, 1, 0, 1, 0},
              {w->b_out, 4, C, 1, 0, 1, 0},
              {w->pre_weight, 4, C, 1, 0, 1, 0},
              {w->pre_bias, 4, C, 1, 0, 1, 0},
              {w->post_weight, 4, C, 1, 0, 1, 0},
              {w->post_bias, 4, C, 1, 0, 1, 0},
              {w->q_weight, 4, 128, 1, 0, 1, 0},
              {w->k_weight, 4, 128, 1, 0, 1, 0},
              {w->freqs, 8, bp->rotary_dim / 2, 1, 0, 1, 0}};
  const Rows taken[2] = {Rows(workspace, 1, static_cast<int64_t>(ws.hi - ws.lo), 1, 0, 1, 0),
                         Rows(out, sx, rows * bp->C, 1, 0, 1, 0)};
  for (const auto& r : read) {
    if (!r.base) continue;
    const Rows in(r.base, r.size, r.row, r.n0, r.s0, r.n1, r.s1);
    if (!apart(taken[0], in) || !apart(taken[1], in)) return BSA_ERR_INVALID;
  }
  BlockWs b;
  block_carve(p, bp->C, static_cast<uint8_t*>(workspace), &b);
  int rc = block_run(p, bp, w, x, out, b, stream, false);
  if (rc) return rc;
  return block_run(p, bp, w, x, out, b, stream, true);
}

}  // extern "C"
