"""The operators around the attention on the GPU against the fp64 oracle.

Tolerances, fixed before the first run.  u = 2^-24 is fp32's rounding, h the output type's half step
(2^-8 bf16, 2^-24 fp32, relative to the value).
  rotary   a value is two products and a sum of inputs of the pair; cos and sin (sincospif) are right to
           about 2 u and their argument to u pi; the norm's square sum of 128 positive terms in a tree of
           depth 8 + 4 and one rsqrt (2 u) give at most 10 u relative.  In all below 2^-20 (|x0| + |x1|) m.
  gate     a sum of C values in chunks of 32 a thread, 5 steps in a warp and up to 32 warps is right to
           70 u of the sum of magnitudes (2^-17.8); a mean square has only positive terms, so the
           factor rsqrt is right to 2^-18; a layer norm's mean is right to 2^-17.8 mean |v|.
  int8     codes and scales are bit-exact (one fp32 division, one product, one rounding); through the
           fused norm a value moves by 2^-17 of the row's largest, so a code is within half a step + that.
  linear   the sum is exact; its conversion, two products and a sum round 4 times: 4 u.
"""

import numpy as np
import pytest
import torch

from block_sparse_video_bsa_b200 import bsa
from oracle import bsa_oracle_block as orb

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rnd(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def host(t):
    return None if t is None else t.double().cpu().numpy()


# ------------------------------------------------------------------ rotary

def check_rotary(got, x, pos, freqs, layout, pairs, weight, eps, scale, inverse=False):
    """got, x [B, H, N, 128] tensors; pos [B or 1, N, axes]."""
    for b in range(x.shape[0]):
        p = host(pos[b if pos.shape[0] > 1 else 0]).astype(np.int64)
        ref = orb.rotary(host(x[b]), p, freqs.cpu().numpy(), layout, pairs, host(weight), eps, scale, inverse)
        src = host(x[b]) if weight is None else orb.rms(host(x[b]), eps) * host(weight)
        r = 2 * len(freqs)
        size = np.abs(src)
        part = size.copy()
        lo = np.arange(r // 2) if layout == "half" else 2 * np.arange(r // 2)
        hi = lo + (r // 2 if layout == "half" else 1)
        part[..., lo] = part[..., hi] = scale * (size[..., lo] + size[..., hi])
        tol = HALF[got.dtype] * np.abs(ref) + 2.0 ** -20 * part
        err = np.abs(host(got[b]) - ref)
        assert (err <= tol).all(), (err - tol).max()


CASES = [
    # B, H, N, r, layout, pairs, norm, in, out
    (1, 1, 1, 128, "half", [64], False, torch.bfloat16, torch.bfloat16),
    (1, 56, 1, 128, "interleaved", [64], True, torch.bfloat16, torch.bfloat16),
    (2, 3, 17, 96, "half", [16, 16, 16], True, torch.bfloat16, torch.bfloat16),
    (1, 5, 131, 96, "interleaved", [16, 16, 16], False, torch.float32, torch.float32),
    (3, 2, 40, 10, "half", [5], True, torch.bfloat16, torch.float32),
    (1, 17, 33, 2, "interleaved", [1], False, torch.float32, torch.bfloat16),
    (1, 4, 9, 120, "half", [20, 20, 20], False, torch.bfloat16, torch.bfloat16),
    (2, 2, 65, 32, "half", [4, 4, 4, 4], True, torch.float32, torch.float32),
    (1, 7, 300, 128, "half", [22, 21, 21], True, torch.bfloat16, torch.bfloat16),
]


@pytest.mark.parametrize("B,H,N,r,layout,pairs,norm,tin,tout", CASES)
def test_rotary_from_a_token_major_projection(cuda_dev, B, H, N, r, layout, pairs, norm, tin, tout):
    qkv = rnd(1, B, N, 3, H, 128, dtype=tin)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    g = torch.Generator(device="cuda").manual_seed(2)
    pos = torch.randint(-1000, 1_000_000, (B, N, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
    freqs, m = bsa.rotary_freqs(pairs, scaling="yarn", factor=4.0, trained_length=4096)
    wq, wk = (1 + rnd(3 + i, 128, scale=0.1) if norm else None for i in range(2))
    keep = qkv.clone()
    Q, K, V = bsa.rotary(q, k, v, pos, freqs, layout, pairs, wq, wk, 1e-6, m, out_dtype=tout)
    assert Q.shape == (B, H, N, 128) and Q.is_contiguous() and Q.dtype == tout
    check_rotary(Q, q, pos, freqs, layout, pairs, wq, 1e-6, m)
    check_rotary(K, k, pos, freqs, layout, pairs, wk, 1e-6, m)
    assert torch.equal(V, v.to(tout))
    assert torch.equal(qkv, keep)


def test_rotary_far_positions(cuda_dev):
    # the ends of int32, where fp32 angles would be off by whole turns
    N = 6
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [2 ** 30 + 7], [1], [0], [-1]], dtype=torch.int32, device="cuda")
    q = rnd(5, 1, 2, N, 128)
    freqs, m = bsa.rotary_freqs(64)
    Q, _, _ = bsa.rotary(q, None, None, pos, freqs)
    # fp64 keeps f to 2^-53: 2^31 of it is 2^-22 of a radian
    ref = orb.rotary(host(q[0]), host(pos).astype(np.int64), freqs.cpu().numpy(), "half", [64])
    assert np.abs(host(Q[0]) - ref).max() <= (2.0 ** -20 + 2.0 ** -21) * 2 * np.abs(host(q)).max()


def test_rotary_in_place_and_inverse(cuda_dev):
    B, H, N = 2, 4, 50
    qkv = rnd(6, B, N, 3, H, 128)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freqs, _ = bsa.rotary_freqs(48)
    views = [qkv[:, :, i].transpose(1, 2) for i in range(3)]
    Q, K, V = bsa.rotary(*views, pos, freqs)
    keep = qkv.clone()
    a = bsa.rotary(*views, pos, freqs, out=views)
    assert a[0].data_ptr() == views[0].data_ptr()
    assert torch.equal(views[0], Q) and torch.equal(views[1], K) and torch.equal(views[2], V)
    back = bsa.rotary(*views, pos, freqs, inverse=True)
    for i in range(3):
        want = keep[:, :, i].transpose(1, 2)
        assert (back[i] - want).abs().max() <= 2.0 ** -19 * 2 * want.abs().max()


def test_rotary_leaves_the_rest_alone(cuda_dev):
    # outputs inside a larger buffer: nothing around them is written; NaN and infinity past rotary_dim pass
    B, H, N = 1, 3, 21
    big = torch.full((B, H, N + 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q = rnd(7, B, H, N, 128, dtype=torch.bfloat16)
    q[..., 100] = float("inf")
    q[..., 127] = float("nan")
    out = big[:, :, 2:2 + N]
    freqs, _ = bsa.rotary_freqs(25)
    for layout in ("half", "interleaved"):
        big.fill_(7.0)
        bsa.rotary(q, None, None, torch.arange(N, dtype=torch.int32, device="cuda"), freqs, layout, out=[out, None, None])
        assert (big[:, :, :2] == 7).all() and (big[:, :, 2 + N:] == 7).all()
        assert torch.equal(out[..., 50:127], q[..., 50:127]) and out[..., 127].isnan().all()
        assert out[..., :50].isfinite().all()


def test_rotary_of_no_dimension_changes_the_layout(cuda_dev):
    qkv = rnd(15, 2, 19, 3, 5, 128, dtype=torch.bfloat16)
    views = [qkv[:, :, i].transpose(1, 2) for i in range(3)]
    pos, freqs = torch.zeros(19, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda")
    for got, want in zip(bsa.rotary(*views, pos, freqs), views):
        assert torch.equal(got, want) and got.is_contiguous()


def test_rotary_positions_of_each_batch_entry_and_broadcast_rows(cuda_dev):
    # strided positions [B, N, axes], and one row of q read for every token (stride 0)
    B, H, N = 3, 2, 37
    pos = torch.randint(0, 5000, (B, N, 4), device="cuda", dtype=torch.int32)[:, :, :3]
    freqs, _ = bsa.rotary_freqs([10, 11, 11])
    q = rnd(16, B, H, 1, 128).expand(B, H, N, 128)
    Q, _, _ = bsa.rotary(q, None, None, pos, freqs, "interleaved", [10, 11, 11])
    check_rotary(Q, q, pos, freqs, "interleaved", [10, 11, 11], None, 0, 1.0)


def test_rotary_other_head_counts_and_streams(cuda_dev):
    q, k, v = rnd(8, 1, 8, 30, 128), rnd(9, 1, 2, 30, 128), rnd(10, 1, 2, 30, 128)
    pos = torch.arange(30, dtype=torch.int32, device="cuda")
    freqs, _ = bsa.rotary_freqs(64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Q, K, V = bsa.rotary(q, k, v, pos, freqs, stream=s)
    s.synchronize()
    check_rotary(Q, q, pos[None, :, None], freqs, "half", [64], None, 0, 1.0)
    check_rotary(K, k, pos[None, :, None], freqs, "half", [64], None, 0, 1.0)
    assert torch.equal(V, v)


# ------------------------------------------------------------------ gate norm

def run_gate_norm(x, y, gate, scale, shift, pre, post, aff, eps, rs=1.0, bs=1.0, **kw):
    C = x.shape[-1]
    ws = [1 + rnd(40 + i, C, scale=0.1) if i % 2 == 0 else rnd(40 + i, C, scale=0.1) for i in range(4)] if aff else [None] * 4
    if y is None:
        ws[2] = ws[3] = None
    h, z = bsa.gate_norm(x, y, gate, scale, shift, pre, ws[0], ws[1], post, ws[2], ws[3], eps, rs, bs, **kw)
    return h, z, ws


def gate_norm_bounds(x, y, gate, scale, shift, pre, post, ws, eps, rs, bs):
    """(h, z, error bound of h, error bound of z) before the output's rounding, from the formulas."""
    full = lambda t: None if t is None else host(t if t.dim() == 3 else (t[:, None] if t.dim() == 2 else t[None, None]))  # noqa: E731
    X, Y, G, S, T = host(x), host(y), full(gate), full(scale), full(shift)
    W = [host(w) for w in ws]
    h, z = orb.gate_norm(X, Y, G, S, T, pre, W[0], W[1], post, W[2], W[3], eps, rs, bs)

    def norm_err(v, e, kind, w, b):
        """Bound of norm(v) when v is off by e: (value, bound)."""
        if kind == "none":
            n, f = v, e
        else:
            c = v - v.mean(-1, keepdims=True) if kind == "layer" else v
            inv = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
            # the mean's own error, then the factor's: rms(e) moves the deviation's root by at most itself
            em = 2.0 ** -17.8 * np.abs(v).mean(-1, keepdims=True) + e.mean(-1, keepdims=True) if kind == "layer" else 0.0
            ee = e + em
            rel = 2.0 ** -18 + np.sqrt((ee * ee).mean(-1, keepdims=True)) * inv
            n, f = c * inv, ee * inv + np.abs(c * inv) * rel
        if w is not None:
            n, f = n * w, f * np.abs(w) + 2.0 ** -23 * np.abs(n * w)
        if b is not None:
            n, f = n + b, f + 2.0 ** -23 * np.abs(n + b)
        return n, f
    eh = np.zeros_like(X)
    if Y is not None:
        n, f = norm_err(Y, np.zeros_like(Y), post, W[2], W[3])
        g = 1.0 if G is None else G
        eh = np.abs(bs * g) * (f + 2.0 ** -22 * np.abs(n)) + 2.0 ** -23 * (np.abs(rs * X) + np.abs(h))
    n, f = norm_err(h, eh, pre, W[0], W[1])
    a = 1.0 if S is None else 1.0 + S
    ez = np.abs(a) * (f + 2.0 ** -22 * np.abs(n)) + 2.0 ** -23 * np.abs(n) + 2.0 ** -23 * np.abs(z)
    return h, z, eh, ez


def close(got, want, bound):
    err = np.abs(host(got) - want)
    tol = bound + HALF[got.dtype] * np.abs(want) + 1e-37
    assert (err <= tol).all(), ((err - tol).max(), np.unravel_index((err - tol).argmax(), err.shape))


GN = [
    # B, N, C, pre, post, x, y, mod, mod shape, affine
    (1, 1, 7168, "rms", "rms", torch.bfloat16, torch.bfloat16, torch.float32, "b", True),
    (2, 5, 256, "layer", "rms", torch.bfloat16, torch.bfloat16, torch.bfloat16, "b1", False),
    (3, 7, 1111, "layer", "layer", torch.float32, torch.bfloat16, torch.bfloat16, "n", True),
    (1, 400, 512, "rms", "none", torch.float32, torch.float32, torch.float32, "n", True),
    (2, 300, 1000, "none", "layer", torch.bfloat16, torch.float32, torch.float32, "c", True),
    (1, 3, 1, "rms", "layer", torch.float32, torch.float32, torch.float32, "b", False),
    (1, 2, 7, "layer", "rms", torch.bfloat16, torch.bfloat16, torch.float32, "b", True),
    (1, 310, 7168, "layer", "rms", torch.bfloat16, torch.bfloat16, torch.float32, "b", False),
    (1, 301, 8200, "rms", "rms", torch.bfloat16, torch.bfloat16, torch.bfloat16, "b", False),
    (1, 300, 16640, "layer", "rms", torch.float32, torch.bfloat16, torch.float32, "b", True),
    (1, 2, 32768, "rms", "layer", torch.bfloat16, torch.bfloat16, torch.float32, "b", True),
    (1, 2, 32767, "layer", "layer", torch.float32, torch.bfloat16, torch.float32, "b", False),
]


@pytest.mark.parametrize("B,N,C,pre,post,tx,ty,tm,shape,aff", GN)
def test_gate_norm(cuda_dev, B, N, C, pre, post, tx, ty, tm, shape, aff):
    x, y = rnd(11, B, N, C, dtype=tx) + 3, rnd(12, B, N, C, dtype=ty) + 1
    s = dict(b=(B, C), b1=(B, 1, C), n=(B, N, C), c=(C,))[shape]
    gate, scale, shift = (rnd(13 + i, *s, dtype=tm, scale=0.5) for i in range(3))
    args = (x, y, gate, scale, shift, pre, post)
    h, z, ws = run_gate_norm(*args, aff, 1e-6, 0.5, 2.0)
    assert h.dtype == tx and z.dtype == torch.bfloat16
    hr, zr, eh, ez = gate_norm_bounds(*args, ws, 1e-6, 0.5, 2.0)
    close(h, hr, eh)
    close(z, zr, ez)
    # fp32 result, and the residual updated in place: the same values
    x2 = x.clone()
    h2, z2, _ = run_gate_norm(x2, *args[1:], aff, 1e-6, 0.5, 2.0, h_out=x2, z_dtype=torch.float32)
    assert h2 is x2 and torch.equal(h2, h) and torch.equal(z2.bfloat16(), z)
    close(z2, zr, ez)
    # the two halves alone
    h3, none, _ = run_gate_norm(x, y, gate, None, None, pre, post, False, 1e-6, want_z=False)
    assert none is None and h3.shape == x.shape
    same, z4, ws4 = run_gate_norm(x, None, None, scale, shift, pre, "none", aff, 1e-6)
    assert same is x
    _, zr4, _, ez4 = gate_norm_bounds(x, None, None, scale, shift, pre, "none", ws4, 1e-6, 1.0, 1.0)
    close(z4, zr4, ez4)


@pytest.mark.parametrize("C", [64, 1111, 7168])
def test_gate_norm_codes(cuda_dev, C):
    B, N = 2, 170
    x, y = rnd(20, B, N, C, dtype=torch.bfloat16), rnd(21, B, N, C, dtype=torch.bfloat16)
    gate, scale, shift = (rnd(22 + i, B, C, scale=0.5) for i in range(3))
    args = (x, y, gate, scale, shift, "layer", "rms")
    h, (codes, top), ws = run_gate_norm(*args, True, 1e-6, quantize=True)
    _, zr, _, ez = gate_norm_bounds(*args, ws, 1e-6, 1.0, 1.0)
    zr, ez = zr.reshape(B * N, C), ez.reshape(B * N, C)
    amax = np.abs(zr).max(1)
    assert codes.shape == (B * N, C) and codes.stride(0) % 16 == 0
    assert (np.abs(host(top) - amax / 127) <= ez.max(1) / 127 + 2.0 ** -23 * amax / 127).all()
    err = np.abs(host(codes) * host(top)[:, None] - zr)
    assert (err <= 0.5 * host(top)[:, None] * (1 + 2.0 ** -16) + 2 * ez.max(1)[:, None]).all()
    assert (codes.abs().amax(1) == 127).all()
    # one source of truth: the codes of the fp32 result are the same codes
    _, z32, _ = run_gate_norm(*args, True, 1e-6, z_dtype=torch.float32)
    c2, t2 = bsa.quantize_int8(z32)
    assert torch.equal(c2, codes) and torch.equal(t2, top)


def test_gate_norm_odd_rows_and_strides(cuda_dev):
    # rows inside wider buffers, at an odd offset: scalar accesses, nothing around them written
    B, N, C = 2, 9, 130
    wide = rnd(30, B, N, C + 7, dtype=torch.bfloat16)
    x, y = wide[..., 3:3 + C], rnd(31, B, N, 2 * C)[..., 1:1 + C]
    buf = torch.full((B, N, C + 6), 9.0, dtype=torch.bfloat16, device="cuda")
    h, z = bsa.gate_norm(x, y, pre="rms", post="rms", h_out=buf[..., 3:3 + C])
    hr, zr, eh, ez = gate_norm_bounds(x, y, None, None, None, "rms", "rms", [None] * 4, 1e-6, 1.0, 1.0)
    close(h, hr, eh)
    close(z, zr, ez)
    assert (buf[..., :3] == 9).all() and (buf[..., 3 + C:] == 9).all()


def test_gate_norm_extreme_rows(cuda_dev):
    C = 512
    x = rnd(32, 1, 6, C)
    x[0, 0] = 0.0                      # nothing: eps keeps it 0
    x[0, 1] = 5.0                      # no deviation: a layer norm gives 0
    x[0, 2] *= 1e-20
    x[0, 3, 7] = float("inf")
    x[0, 4, 9] = float("nan")
    x[0, 5] += 1e4                     # large mean, small deviation
    for pre in ("rms", "layer"):
        _, z = bsa.gate_norm(x, pre=pre, z_dtype=torch.float32)
        rows = [0, 1, 2, 5]
        _, zr, _, ez = gate_norm_bounds(x[:, rows], None, None, None, None, pre, "none", [None] * 4, 1e-6, 1.0, 1.0)
        close(z[:, rows], zr, ez)
        assert not z[0, 3].isfinite().all() and z[0, 4].isnan().all()
        _, (codes, top) = bsa.gate_norm(x, pre=pre, quantize=True)
        assert top[[3, 4]].isnan().all() and not codes[[3, 4]].any() and top[[0, 1, 2, 5]].isfinite().all()


# ------------------------------------------------------------------ int8 rows and product

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7168), (3, 17), (300, 7168), (400, 1111), (2, 32768), (299, 28672), (1, 32767), (500, 256)])
def test_quantize_int8_is_bit_exact(cuda_dev, M, K, dtype):
    x = rnd(50, M, K, dtype=dtype) * (1 + 9 * (rnd(51, K) > 2)).to(dtype)
    codes, scale = bsa.quantize_int8(x)
    c, s = orb.quantize_int8(x.float().cpu().numpy())
    assert (codes.cpu().numpy() == c).all() and (scale.cpu().numpy() == s).all()


def test_quantize_int8_rows_of_special_values(cuda_dev):
    x = rnd(52, 8, 100, dtype=torch.bfloat16)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 99] = float("nan")
    x[3] *= 1e-37
    x[4] = 3e38
    x[5, 0] = -float("inf")
    codes, scale = bsa.quantize_int8(x)
    c, s = orb.quantize_int8(x.float().cpu().numpy())
    assert (codes.cpu().numpy() == c).all() and np.array_equal(scale.cpu().numpy(), s, equal_nan=True)


@pytest.mark.parametrize("B,H,N", [(1, 56, 130), (2, 3, 33), (1, 1, 1)])
def test_quantize_int8_of_head_major_rows(cuda_dev, B, H, N):
    O = rnd(53, B, H, N, 128, dtype=torch.bfloat16)
    codes, scale = bsa.quantize_int8(O)
    flat = O.permute(0, 2, 1, 3).reshape(B * N, H * 128)
    c, s = bsa.quantize_int8(flat)
    assert torch.equal(codes, c) and torch.equal(scale, s)
    odd = rnd(54, B, H, N, 129)[..., 1:]          # rows that start on no boundary, a segment of 128
    c, s = bsa.quantize_int8(odd)
    c2, s2 = bsa.quantize_int8(odd.permute(0, 2, 1, 3).reshape(B * N, H * 128))
    assert torch.equal(c, c2) and torch.equal(s, s2)


def codes_of(seed, M, K):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((M, -(-K // 16) * 16), 77, dtype=torch.int8, device="cuda")   # what lies past K must not count
    buf[:, :K] = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    return buf[:, :K]


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 7168, 7168), (3, 200, 300), (16, 129, 1111), (17, 256, 128), (33, 515, 1111), (64, 1000, 515),
          (65, 130, 640), (127, 128, 4096), (128, 128, 128), (129, 257, 129), (255, 512, 1000), (256, 256, 256), (257, 513, 16), (300, 40, 7168),
          (513, 1030, 2049), (1000, 515, 1111), (1500, 2304, 900), (2, 21504, 640), (40, 7168, 28672), (700, 16, 32768)]


def check_linear(M, N, K, out_dtype, bias, seed=60, out=None):
    a, w = codes_of(seed, M, K), codes_of(seed + 1, N, K)
    sa, sw = rnd(seed + 2, M).abs() + 0.01, rnd(seed + 3, N).abs() + 0.01
    b = rnd(seed + 4, N, scale=100.0) if bias else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bsa.linear_int8(a, sa, w, sw, b, out_dtype, out, status)
    # the whole sum in fp64: products of at most 127^2, fewer than 2^15 of them, are exact
    total = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    ref = total if b is None else total + b.double()
    tol = HALF[got.dtype] * ref.abs() + 4 * 2.0 ** -24 * (total.abs() + (0 if b is None else b.double().abs()))
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()
    assert int(status) == 0
    return got


@pytest.mark.parametrize("out_dtype,bias", [(torch.bfloat16, True), (torch.float32, False)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_int8(cuda_dev, M, N, K, out_dtype, bias):
    check_linear(M, N, K, out_dtype, bias)


def test_linear_int8_rows_of_a_wider_output(cuda_dev):
    for M, N, K in ((5, 77, 100), (300, 130, 200), (600, 333, 64)):
        for dtype in (torch.bfloat16, torch.float32):
            buf = torch.full((M + 2, N + 9), 5.0, dtype=dtype, device="cuda")
            check_linear(M, N, K, dtype, True, out=buf[1:1 + M, 4:4 + N])
            assert (buf[0] == 5).all() and (buf[-1] == 5).all() and (buf[:, :4] == 5).all() and (buf[:, 4 + N:] == 5).all()


def test_linear_int8_largest_sums(cuda_dev):
    # every product 127^2 of the longest rows: 2^15 127^2 < 2^31 stays exact
    for M in (2, 300):
        a = torch.full((M, 32768), 127, dtype=torch.int8, device="cuda")
        w = torch.full((40, 32768), -127, dtype=torch.int8, device="cuda")
        one = torch.ones(300, device="cuda")
        out = bsa.linear_int8(a, one[:M], w, one[:40], out_dtype=torch.float32)
        assert (out == float(np.float32(-127 * 127 * 32768))).all()


def test_linear_int8_marks_rows_without_a_scale(cuda_dev):
    x = rnd(70, 40, 256)
    x[7, 3] = float("nan")
    a, sa = bsa.quantize_int8(x)
    w, sw = bsa.quantize_int8(rnd(71, 30, 256))
    out = bsa.linear_int8(a, sa, w, sw)
    assert out[7].isnan().all() and out[:7].isfinite().all() and out[8:].isfinite().all()


# ------------------------------------------------------------------ together, and as graphs

def test_calls_are_deterministic_and_captured(cuda_dev):
    B, N, H, C = 1, 200, 4, 512
    x, y = rnd(80, B, N, C, dtype=torch.bfloat16), rnd(81, B, N, C, dtype=torch.bfloat16)
    gate, scale, shift = (rnd(82 + i, B, C) for i in range(3))
    w, sw = bsa.quantize_int8(rnd(85, 3 * H * 128, C))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freqs, m = bsa.rotary_freqs(64)
    one = 1 + rnd(86, 128, scale=0.1)

    def step():
        h, (a, sa) = bsa.gate_norm(x, y, gate, scale, shift, post="rms", quantize=True)
        qkv = bsa.linear_int8(a, sa, w, sw).view(B, N, 3, H, 128)
        Q, K, V = bsa.rotary(*(qkv[:, :, i].transpose(1, 2) for i in range(3)), pos, freqs, q_weight=one, k_weight=one)
        O = bsa.forward(Q, K, V, 1)
        return (h, Q, K, V, O, *bsa.quantize_int8(O))

    first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for g, outs in graphs:
        g.replay()
    for g, outs in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, outs in graphs:
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ many rows (the streamed kernel)

RING = [
    # B, N, C, pre, post, x, y, mod shape, affine
    (1, 700, 7168, "layer", "rms", torch.bfloat16, torch.bfloat16, "b", True),
    (2, 400, 2056, "rms", "layer", torch.bfloat16, torch.float32, "b1", True),
    (3, 333, 1032, "layer", "none", torch.float32, torch.bfloat16, "c", False),
    (1, 601, 1024, "none", "rms", torch.float32, torch.float32, "c", False),
    (150, 5, 2048, "rms", "rms", torch.bfloat16, torch.bfloat16, "b", True),
    (1, 593, 12288, "layer", "none", torch.bfloat16, torch.bfloat16, "c", False),
    (1, 2500, 7168, "layer", "rms", torch.bfloat16, torch.bfloat16, "n", True),
    (2, 2700, 520, "rms", "layer", torch.float32, torch.bfloat16, "n", True),
    (1, 13000, 256, "layer", "rms", torch.bfloat16, torch.bfloat16, "n", False),
    (1, 13003, 136, "rms", "rms", torch.bfloat16, torch.bfloat16, "b", True),
    # two stages, fewer than the groups of warps that a CTA has room for
    (2, 1000, 6992, "rms", "layer", torch.bfloat16, torch.bfloat16, "nf", False),
    (1, 2000, 4816, "none", "rms", torch.float32, torch.float32, "nf", False),
]


@pytest.mark.parametrize("B,N,C,pre,post,tx,ty,shape,aff", RING)
def test_gate_norm_of_many_rows(cuda_dev, B, N, C, pre, post, tx, ty, shape, aff):
    x, y = rnd(90, B, N, C, dtype=tx) + 3, rnd(91, B, N, C, dtype=ty) - 2
    s = dict(b=(B, C), b1=(B, 1, C), c=(C,), n=(B, N, C), nf=(B, N, C))[shape]
    gate, scale, shift = (rnd(92 + i, *s, dtype=torch.float32 if shape == "nf" else torch.bfloat16, scale=0.5) for i in range(3))
    args = (x, y, gate, scale, shift, pre, post)
    h, z, ws = run_gate_norm(*args, aff, 1e-6, 0.5, 2.0)
    hr, zr, eh, ez = gate_norm_bounds(*args, ws, 1e-6, 0.5, 2.0)
    close(h, hr, eh)
    close(z, zr, ez)
    _, (codes, top), _ = run_gate_norm(*args, aff, 1e-6, 0.5, 2.0, quantize=True)
    err = np.abs(host(codes).reshape(zr.shape) * host(top).reshape(B, N, 1) - zr)
    assert (err <= 0.5 * host(top).reshape(B, N, 1) * (1 + 2.0 ** -16) + 2 * ez.max(-1, keepdims=True)).all()
    x2 = x.clone()
    h2, z2, _ = run_gate_norm(x2, *args[1:], aff, 1e-6, 0.5, 2.0, h_out=x2, z_dtype=torch.float32)
    assert torch.equal(h2, h) and torch.equal(z2.bfloat16(), z)
    # each part left out
    _, z3, ws3 = run_gate_norm(x, None, None, scale, None, pre, "none", aff, 1e-6)
    _, zr3, _, ez3 = gate_norm_bounds(x, None, None, scale, None, pre, "none", ws3, 1e-6, 1.0, 1.0)
    close(z3, zr3, ez3)
    h4, none, ws4 = run_gate_norm(x, y, None, None, None, pre, post, False, 1e-6, want_z=False)
    hr4, _, eh4, _ = gate_norm_bounds(x, y, None, None, None, pre, post, ws4, 1e-6, 1.0, 1.0)
    assert none is None
    close(h4, hr4, eh4)


@pytest.mark.parametrize("N", [20, 1300])
def test_gate_norm_without_a_branch_ignores_its_norm(cuda_dev, N):
    x, w = rnd(98, 1, N, 2048, dtype=torch.bfloat16), rnd(99, 2048)
    _, a = bsa.gate_norm(x, post="layer", post_weight=w, post_bias=w)
    _, b = bsa.gate_norm(x)
    assert torch.equal(a, b)


@pytest.mark.parametrize("N,C,dtype", [(23567, 2552, torch.float32), (37740, 1024, torch.bfloat16), (30000, 512, torch.bfloat16), (20000, 5120, torch.bfloat16)])
def test_gate_norm_streams_rows_in_order(cuda_dev, N, C, dtype):
    # without norms nothing but the stages' barriers holds the groups of warps together: every value is exact,
    # over many calls
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, y = rnd(100, 1, N, C, dtype=dtype), rnd(101, 1, N, C, dtype=torch.bfloat16)
    want = (x.float() + y.float()).to(dtype)
    for _ in range(40):
        h, z = bsa.gate_norm(x, y, pre="none", post="none", dev_status=status)
        assert torch.equal(h, want) and torch.equal(z, (x.float() + y.float()).bfloat16())
    assert int(status) == 0


def test_gate_norm_reports_no_expired_wait(cuda_dev):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = rnd(97, 1, 3000, 2048, dtype=torch.bfloat16)
    _, a = bsa.gate_norm(x)
    _, b = bsa.gate_norm(x, dev_status=status)
    assert torch.equal(a, b) and int(status) == 0


def test_gate_norm_of_many_rows_in_wider_buffers(cuda_dev):
    # rows of a wider buffer and a NaN row: neighbours of both are untouched
    B, N, C = 2, 400, 2048
    x, y = rnd(95, B, N, C + 64)[..., 32:32 + C], rnd(96, B, N, C)
    y[1, 7, 5] = float("nan")
    buf = torch.full((B, N, C + 16), 3.0, device="cuda")
    h, z = bsa.gate_norm(x, y, pre="layer", post="rms", h_out=buf[..., 8:8 + C])
    assert (buf[..., :8] == 3).all() and (buf[..., 8 + C:] == 3).all()
    assert z[1, 7].isnan().all() and h[1, 7].isnan().all()
    keep = torch.ones(B, N, dtype=torch.bool, device="cuda")
    keep[1, 7] = False
    hr, zr, eh, ez = gate_norm_bounds(x[keep][None], y[keep][None], None, None, None, "layer", "rms", [None] * 4, 1e-6, 1.0, 1.0)
    close(h[keep][None], hr, eh)
    close(z[keep][None], zr, ez)


# ------------------------------------------------------------------ the block path

def block_case(B, N, H, C, seed, dtype=torch.bfloat16):
    r = lambda i, *s, **k: rnd(seed + i, *s, **k)  # noqa: E731
    w_qkv, s_qkv = bsa.quantize_int8(r(0, 3 * H * 128, C, scale=C ** -0.5))
    w_out, s_out = bsa.quantize_int8(r(1, C, H * 128, scale=(H * 128) ** -0.5))
    pos = torch.stack((torch.arange(N) // 24, torch.arange(N) // 6 % 4, torch.arange(N) % 6), 1).to(torch.int32).cuda()
    freqs, m = bsa.rotary_freqs([22, 21, 21])
    return dict(x=r(2, B, N, C, dtype=dtype), w_qkv=w_qkv, s_qkv=s_qkv, w_out=w_out, s_out=s_out, positions=pos, freqs=freqs, rope_scale=m,
                gate=r(3, B, C), scale=r(4, B, C, scale=0.3), shift=r(5, B, C, scale=0.3), b_qkv=r(6, 3 * H * 128, scale=0.1),
                b_out=r(7, C, scale=0.1), pre="layer", post="rms", post_weight=1 + r(8, C, scale=0.1), q_weight=1 + r(9, 128, scale=0.1),
                k_weight=1 + r(10, 128, scale=0.1), layout="interleaved", axis_pairs=[22, 21, 21])


def by_steps(c, top_k, prefix, variant):
    B, N, C = c["x"].shape
    H = c["w_out"].shape[1] // 128
    _, (a, sa) = bsa.gate_norm(c["x"], scale=c["scale"], shift=c["shift"], pre=c["pre"], quantize=True)
    qkv = bsa.linear_int8(a, sa, c["w_qkv"], c["s_qkv"], c["b_qkv"]).view(B, N, 3, H, 128)
    Q, K, V = bsa.rotary(*(qkv[:, :, i].transpose(1, 2) for i in range(3)), c["positions"], c["freqs"], c["layout"], c["axis_pairs"],
                         c["q_weight"], c["k_weight"], 1e-6, c["rope_scale"])
    O = bsa.forward(Q, K, V, top_k, prefix, variant)
    y = bsa.linear_int8(*bsa.quantize_int8(O), c["w_out"], c["s_out"], c["b_out"]).view(B, N, C)
    h, _ = bsa.gate_norm(c["x"], y, c["gate"], post=c["post"], post_weight=c["post_weight"], want_z=False)
    return h


@pytest.mark.parametrize("B,N,H,C,top_k,prefix,variant,dtype", [
    (1, 1, 1, 128, 1, 0, "anchor", torch.bfloat16), (2, 300, 3, 200, 1, 0, "mean", torch.bfloat16),
    (1, 700, 2, 1111, 2, 128, "anchor", torch.float32), (1, 1500, 5, 640, 3, 0, "anchor", torch.bfloat16)])
def test_forward_block_is_its_steps(cuda_dev, B, N, H, C, top_k, prefix, variant, dtype):
    c = block_case(B, N, H, C, 200, dtype)
    want = by_steps(c, top_k, prefix, variant)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bsa.forward_block(**c, top_k=top_k, prefix=prefix, variant=variant, dev_status=status)
    assert torch.equal(got, want) and int(status) == 0
    x = c["x"].clone()                   # the residual stream updated in place
    assert bsa.forward_block(**dict(c, x=x), top_k=top_k, prefix=prefix, variant=variant, out=x) is x
    assert torch.equal(x, want)


def test_forward_block_against_the_oracles(cuda_dev):
    """Every key block listed, so the attention is dense and exact.  The int8 rows of z are those of the oracle up
    to ties; q, k, v, O and y are bf16 (2^-9 of a value each, in the mean), the attention's own bound is 1e-2, and
    an O that is off by e moves the codes of a share e / step of its values by a step of 1/40 of the deviation:
    sqrt(0.025 * 0.005), about 1e-2.  Together below 3e-2 of what the block adds to x."""
    B, N, H, C = 1, 260, 2, 320
    c = block_case(B, N, H, C, 300, torch.float32)
    out = bsa.forward_block(**c, top_k=3)
    n = {k: host(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    _, z = orb.gate_norm(n["x"], scale=n["scale"][:, None], shift=n["shift"][:, None], pre="layer")
    a, sa = orb.quantize_int8(z[0])
    qkv = orb.linear_int8(a, sa, n["w_qkv"], n["s_qkv"].astype(np.float32), n["b_qkv"]).reshape(N, 3, H, 128).transpose(1, 2, 0, 3)
    pos = n["positions"].astype(np.int64)
    q, k = (orb.rotary(qkv[i], pos, n["freqs"], "interleaved", [22, 21, 21], n[w], 1e-6, 1.0) for i, w in ((0, "q_weight"), (1, "k_weight")))
    s = q @ k.transpose(0, 2, 1) / np.sqrt(128)
    pr = np.exp(s - s.max(-1, keepdims=True))
    O = (pr / pr.sum(-1, keepdims=True)) @ qkv[2]
    o8, so = orb.quantize_int8(O.transpose(1, 0, 2).reshape(N, H * 128))
    y = orb.linear_int8(o8, so, n["w_out"], n["s_out"].astype(np.float32), n["b_out"])
    h, _ = orb.gate_norm(n["x"][0], y, n["gate"], pre="none", post="rms", post_weight=n["post_weight"])
    added, want = host(out[0]) - n["x"][0], h - n["x"][0]
    assert np.linalg.norm(added - want) <= 3e-2 * np.linalg.norm(want)


def test_two_streams_at_once(cuda_dev):
    # the same calls on two streams with their own workspaces: nothing of one shows in the other
    cs = [block_case(1, 900, 3, 512, s) for s in (400, 500)]
    want = [by_steps(c, 2, 0, "anchor") for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            got[i].append(bsa.forward_block(**c, top_k=2, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("B,N,C", [(1, 20_000, 7_168), (2, 700, 2_048), (1, 3_000, 1_111), (1, 1, 7_168), (3, 40, 65)])
def test_gate_norm_codes_are_those_of_its_rows(cuda_dev, B, N, C, token):
    # quantised in the same pass or afterwards from fp32: the same codes and scales, to the bit
    if token and N * C > 10_000_000:
        N //= 8
    x = rnd(600, B, N, C, dtype=torch.bfloat16)
    mod = [0.3 * rnd(601 + i, B, N if token else 1, C) for i in range(2)]
    for pre in ("rms", "layer"):
        _, z = bsa.gate_norm(x, None, None, *mod, pre=pre, z_dtype=torch.float32)
        _, (codes, top) = bsa.gate_norm(x, None, None, *mod, pre=pre, quantize=True)
        want, scale = bsa.quantize_int8(z.reshape(B * N, C))
        assert torch.equal(top, scale)
        assert torch.equal(codes.reshape(B * N, C), want)


@pytest.mark.parametrize("N", [2, 1_000])
def test_gate_norm_sum_of_squares_past_fp32(cuda_dev, N):
    # the mean square overflows: the factor is 0 and z the shift, but for infinities themselves
    C = 7_168
    x = rnd(610, 1, N, C)
    x[0, 0] = 1e25
    x[0, 1, 5] = float("inf")
    shift = rnd(611, 1, 1, C)
    _, z = bsa.gate_norm(x, shift=shift, pre="rms", z_dtype=torch.float32)
    assert torch.equal(z[0, 0], shift[0, 0])
    rest = torch.arange(C, device=z.device) != 5
    assert torch.equal(z[0, 1, rest], shift[0, 0, rest]) and z[0, 1, 5].isnan()


@pytest.mark.parametrize("M,C,H", [(1, 512, 2), (1, 7_168, 56), (40, 1_111, 3), (300, 512, 4), (5_000, 640, 2)])
def test_calls_in_a_row_see_each_other(cuda_dev, M, C, H):
    # launches overlap their starts with the call before: every value a call reads is written by that one or by the caller, again and
    # again into the same places, and nothing may be read early or written over late
    x0 = rnd(700, 1, M, C)
    w1, s1 = bsa.quantize_int8(rnd(701, 3 * H * 128, C))
    w2, s2 = bsa.quantize_int8(rnd(702, C, H * 128))
    pos = torch.arange(M, dtype=torch.int32, device=x0.device)
    freqs, _ = bsa.rotary_freqs(64)
    qkv = torch.empty(M, 3 * H * 128, dtype=torch.bfloat16, device=x0.device)
    heads = torch.empty(1, H, M, 128, dtype=torch.bfloat16, device=x0.device)
    y = torch.empty(M, C, dtype=torch.bfloat16, device=x0.device)

    def chain(x, wait):
        for _ in range(6):
            _, (a, sa) = bsa.gate_norm(x, pre="rms", quantize=True)
            wait()
            bsa.linear_int8(a, sa, w1, s1, out=qkv)
            wait()
            q = qkv.view(1, M, 3, H, 128)[:, :, 0].transpose(1, 2)
            bsa.rotary(q, None, None, pos, freqs, out=(heads, None, None))
            wait()
            a, sa = bsa.quantize_int8(heads)
            wait()
            bsa.linear_int8(a, sa, w2, s2, out=y)
            wait()
            bsa.gate_norm(x, y[None], post="rms", h_out=x, want_z=False)
            wait()
            x.mul_(0.5)
            wait()
        return x

    want = chain(x0.clone(), torch.cuda.synchronize)
    for _ in range(10):
        assert torch.equal(chain(x0.clone(), lambda: None), want)
    x = x0.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        chain(x, lambda: None)
    for _ in range(3):
        x.copy_(x0)
        graph.replay()
        assert torch.equal(x, want)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [(512, 256, 7_168), (2_048, 128, 7_168), (100, 144, 10_001), (128, 640, 11_840), (70, 17, 13_016), (300, 256, 7_000),
                                   (130, 1_000, 13_999), (256, 130, 9_472), (600, 96, 16_000)])
def test_linear_int8_tiles_of_every_width(cuda_dev, M, K, N, out):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    ld = -(-K // 16) * 16
    a, w = [torch.randint(-127, 128, (r, ld), generator=g, device="cuda", dtype=torch.int8)[:, :K] for r in (M, N)]
    sa, sw = [torch.rand(r, generator=g, device="cuda") + 0.1 for r in (M, N)]
    bias = torch.randn(N, generator=g, device="cuda")
    got = bsa.linear_int8(a, sa, w, sw, bias=bias, out_dtype=out).double()
    scaled = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()
    want = scaled + bias.double()
    # the sum (exact below 2^24), its product with a_scale, the fused step and the last rounding: half a step each
    room = 2.0**-23 * scaled.abs() + 2.0**-24 * want.abs() + torch.finfo(out).eps / 2 * (want.abs() + 2.0**-22 * scaled.abs()) + 1e-30
    assert ((got - want).abs() <= room).all()


@pytest.mark.parametrize("N,C", [(3, 512), (2, 7_168), (3, 1_111), (2, 24_000), (3_000, 7_168), (40_000, 264)])
def test_layer_norm_of_rows_far_from_zero(cuda_dev, N, C):
    # the square of the mean is past fp32, the deviations are not
    x = 1e20 + 1e17 * rnd(820, 1, N, C)
    _, z = bsa.gate_norm(x, pre="layer", z_dtype=torch.float32)
    assert z.isfinite().all()
    rows = [0, 1, N - 1]
    _, zr, _, ez = gate_norm_bounds(x[:, rows], None, None, None, None, "layer", "none", [None] * 4, 1e-6, 1.0, 1.0)
    close(z[:, rows], zr, ez)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("N,C", [(3, 512), (1, 8_192), (3_000, 8_192), (40_000, 256), (2_000, 2_048)])
def test_layer_norm_of_one_large_value(cuda_dev, N, C, post):
    # sums of a power of two are exact, so there is no deviation and z is 0, although the value over the smallest
    # root (10^7 times it) is past fp32
    x = torch.full((1, N, C), 2.0 ** 110, device="cuda")
    if post:
        h, z = bsa.gate_norm(torch.zeros_like(x), x, pre="none", post="layer", eps=1e-14, z_dtype=torch.float32)
        assert not h.any()
    else:
        _, z = bsa.gate_norm(x, pre="layer", eps=1e-14, z_dtype=torch.float32)
    assert not z.any()


@pytest.mark.parametrize("B,N,C", [(1, 1, 7_168), (3, 40, 1_111), (2, 700, 2_048), (1, 5_000, 640)])
def test_vectors_made_by_the_call_before(cuda_dev, B, N, C):
    # gate, scale and shift come from a projection and the weights, scales and biases from norms, over and over into the same
    # places, and are read by the very next call
    x, y = rnd(830, B, N, C), rnd(831, B, N, C)
    emb = rnd(832, 1, B, 256)
    w, sw = bsa.quantize_int8(rnd(833, 3 * C, 256))
    mod, w128 = torch.empty(B, 3 * C, device="cuda"), torch.empty(1, 1, 128, device="cuda")
    wa, sa = bsa.quantize_int8(rnd(834, 128, C, scale=C ** -0.5))
    ones = torch.ones(128, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freqs, _ = bsa.rotary_freqs(64)

    def chain(wait):
        e, outs = emb.clone(), []
        for i in range(6):
            _, (a, s) = bsa.gate_norm(e, quantize=True)
            wait()
            bsa.linear_int8(a, s, w, sw, out=mod)
            wait()
            gate, scale, shift = (mod[:, j * C:(j + 1) * C] for j in range(3))
            _, (a, s) = bsa.gate_norm(x, y, gate, scale, shift, post="rms", quantize=True)
            wait()
            q = bsa.linear_int8(a, s, wa, sa, ones, torch.float32)
            wait()
            q = q.view(B, N, 1, 128).transpose(1, 2)
            h, _ = bsa.gate_norm(q[:1, 0, :1], q[:1, 0, -1:], h_out=w128, pre="none", post="rms", want_z=False)
            wait()
            Q, _, _ = bsa.rotary(q, None, None, pos, freqs, q_weight=w128.view(128))
            wait()
            h, z = bsa.gate_norm(Q[:1, 0], pre="rms", pre_weight=w128.view(128), pre_bias=w128.view(128), z_dtype=torch.float32)
            wait()
            outs += [mod.clone(), w128.clone(), Q, z]
            e = e * 0.5 + Q[:, 0, 0, :1].reshape(1, B, 1)
        return outs

    want = chain(torch.cuda.synchronize)
    for _ in range(10):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("form", ["scale", "shift", "both", "both a token", "weight and bias", "gate", "gate a token"])
@pytest.mark.parametrize("C,N,dtype", [(7_168, 4_000, torch.bfloat16), (2_048, 4_000, torch.float32), (256, 30_000, torch.bfloat16)])
def test_gate_norm_rounds_the_same_for_few_and_many_rows(cuda_dev, C, N, dtype, form):
    # without a norm there is no sum to order: the streamed kernel and the other one round every product and every sum
    x, y = rnd(840, 1, N, C, dtype=dtype), rnd(841, 1, N, C, dtype=torch.bfloat16)
    token = "token" in form
    m = [rnd(842 + i, 1, N if token else 1, C, scale=0.3) for i in range(3)]
    w, b = 1 + rnd(845, C, scale=0.1), rnd(846, C, scale=0.1)
    f = x.float()

    def call(rows, **kw):
        v = [t[:, :rows] for t in m]
        if "gate" in form:
            return bsa.gate_norm(x[:, :rows], y[:, :rows], v[0], pre="none", **kw)
        if "weight" in form:
            return bsa.gate_norm(x[:, :rows], pre="none", pre_weight=w, pre_bias=b, **kw)
        return bsa.gate_norm(x[:, :rows], None, None, None if form == "shift" else v[0], None if form == "scale" else v[1], "none", **kw)
    want = {"gate": lambda: f + y.float() * m[0], "weig": lambda: f * w + b, "scal": lambda: f * (1 + m[0]), "shif": lambda: f + m[1],
            "both": lambda: f * (1 + m[0]) + m[1]}[form[:4]]()
    _, few = call(4, z_dtype=torch.float32)
    _, many = call(N, z_dtype=torch.float32)
    assert torch.equal(many, want) and torch.equal(few, want[:, :4])
    _, (codes, top) = call(N, quantize=True)
    c, t = bsa.quantize_int8(want[0])
    assert torch.equal(codes, c) and torch.equal(top, t)
    _, (codes, top) = call(4, quantize=True)
    assert torch.equal(codes, c[:4]) and torch.equal(top, t[:4])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,C", [(4, 7_168), (4_000, 7_168), (4_000, 2_048), (30_000, 256), (3_000, 1_111)])
def test_gate_norm_codes_of_special_rows(cuda_dev, N, C, dtype):
    # rows that hold a NaN or an infinity, at a row's first, last and cut chunks; nothing of them shows in their neighbours
    x = rnd(850, 1, N, C, dtype=dtype)
    keep = x.clone()
    bad = {0: (0, float("nan")), 1: (C - 1, float("inf")), N // 2: (C // 2, -float("inf")), N - 1: (C - 1, float("nan"))}
    for row, (at, v) in bad.items():
        x[0, row, at] = v
    zero = [r for r in (2, N // 2 + 1, N - 3) if r not in bad][:1]
    x[0, zero] = 0
    keep[0, zero] = 0
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[list(bad)] = False
    for pre in ("none", "rms", "layer"):
        _, (codes, top) = bsa.gate_norm(x, pre=pre, quantize=True)
        assert top[~rest].isnan().all() and not codes[~rest].any()
        _, (c, t) = bsa.gate_norm(keep, pre=pre, quantize=True)
        assert torch.equal(codes[rest], c[rest]) and torch.equal(top[rest], t[rest]) and t.isfinite().all()
        assert not c[zero].any() and (t[zero] == np.float32(2.0 ** -100 / 127)).all()


@pytest.mark.parametrize("N,C", [(3, 7_168), (4_000, 7_168), (4_000, 1_111), (30_000, 256)])
def test_gate_norm_codes_differ_from_64_bits_at_borders_only(cuda_dev, N, C):
    """The factor is right to 2^-18 (above) and enters the row's largest value too; product, sum, scale and code product round
    once each: 127 (2^-17 + 8 2^-24), below 127 2^-16 of a code.  So a code is that of 64 bits, or the other one of a border
    that the 64-bit value is this near to."""
    x = (rnd(860, 1, N, C) * (1 + 9 * (rnd(861, C) > 2))).bfloat16()
    scale, shift = (rnd(862 + i, 1, 1, C, scale=0.3) for i in range(2))
    _, (codes, _) = bsa.gate_norm(x, None, None, scale, shift, quantize=True)
    z = x[0].double()
    z = z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    z = z * (1 + scale[0].double()) + shift[0].double()
    exact = z * (127.0 / z.abs().amax(1, keepdim=True))
    off = (codes.double() - exact).abs()
    assert bool((off <= 0.5 + 127 * 2.0 ** -16).all())
    assert bool(((codes.double() == exact.round()) | ((exact - exact.floor() - 0.5).abs() <= 127 * 2.0 ** -16)).all())


def test_captured_over_two_streams_that_join(cuda_dev):
    # a graph whose branches fork and join around the calls: launches that start early wait for both sides
    c = block_case(1, 700, 3, 512, 870)
    B, N, C = c["x"].shape
    H = c["w_out"].shape[1] // 128
    freqs, pos = c["freqs"], c["positions"]
    x = c["x"].clone()

    def step(side):
        main = torch.cuda.current_stream()
        _, (a, sa) = bsa.gate_norm(x, scale=c["scale"], shift=c["shift"], pre="layer", quantize=True)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kv = bsa.linear_int8(a, sa, c["w_qkv"][H * 128:], c["s_qkv"][H * 128:]).view(B, N, 2, H, 128)
            _, K, V = bsa.rotary(None, kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2), pos, freqs, "interleaved", [22, 21, 21])
        q = bsa.linear_int8(a, sa, c["w_qkv"][:H * 128], c["s_qkv"][:H * 128]).view(B, N, H, 128)
        Q, _, _ = bsa.rotary(q.transpose(1, 2), None, None, pos, freqs, "interleaved", [22, 21, 21])
        main.wait_stream(side)
        _, z = bsa.gate_norm(Q.view(1, -1, 128), V.view(1, -1, 128), gate=K.view(1, -1, 128), pre="none")
        codes, s = bsa.quantize_int8(z.view(B, H, N, 128))
        for t in (a, sa, kv, K, V):
            t.record_stream(side)
        return Q, K, V, z, codes, s

    want = [t.clone() for t in step(torch.cuda.current_stream())]
    torch.cuda.synchronize()
    graph, stream, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        got = step(side)
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_from_two_threads(cuda_dev):
    import threading
    cs = [block_case(1, n, 3, 512, 880 + n) for n in (300, 700)]
    want = [by_steps(c, 2, 0, "anchor") for c in cs]
    torch.cuda.synchronize()
    right = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            right.extend([torch.equal(by_steps(cs[i], 2, 0, "anchor"), want[i]) for _ in range(10)])
    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert right == [True] * 40


@pytest.mark.parametrize("norm", [False, True])
def test_rotary_of_several_layouts_in_one_call(cuda_dev, norm):
    # grouped heads of one packed projection, other types, one of the three in place: the bits of a call for each
    B, N, H, G = 2, 75, 6, 2
    buf = rnd(890, B, N, H + 2 * G, 128, dtype=torch.bfloat16)
    q, k = buf[:, :, :H].transpose(1, 2), buf[:, :, H:H + G].transpose(1, 2)
    v = rnd(891, B, G, N, 128)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 977
    freqs, m = bsa.rotary_freqs(40)
    wq, wk = (1 + rnd(892 + i, 128, scale=0.1) if norm else None for i in range(2))
    kw = dict(layout="interleaved", eps=1e-5, scale=m)
    want = (bsa.rotary(q, None, None, pos, freqs, q_weight=wq, **kw)[0], bsa.rotary(None, k, None, pos, freqs, k_weight=wk, **kw)[1], v.clone())
    check_rotary(want[1], k, pos[None, :, None], freqs, "interleaved", [40], wk, 1e-5, m)
    got = bsa.rotary(q, k, v, pos, freqs, q_weight=wq, k_weight=wk, **kw)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)
    K = torch.empty(B, G, N, 128, device="cuda")
    rest = buf[:, :, H:].clone()
    got = bsa.rotary(q, k, v, pos, freqs, q_weight=wq, k_weight=wk, out=(q, K, v), **kw)      # in place: q and v
    assert torch.equal(q, want[0]) and torch.equal(K.bfloat16(), want[1]) and torch.equal(v, want[2])
    assert torch.equal(buf[:, :, H:], rest)
    keep = buf.clone()
    with pytest.raises(bsa.BsaError):      # k's output over q's rows, which another launch turns
        bsa.rotary(q, k, v, pos, freqs, out=(None, buf[:, :, :G].transpose(1, 2), None), **kw)
    assert torch.equal(buf, keep)
