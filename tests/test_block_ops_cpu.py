"""The operators around the attention without a GPU: the oracle against independent forms, the host-side
frequency helper, and the refusals that come before any launch."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from block_sparse_video_bsa_b200 import bsa
from oracle import bsa_oracle_block as orb


# ------------------------------------------------------------------ oracle pins

def test_turns_reduce_far_positions_exactly():
    # sin(p) of whole radians far out, against known identities: angle addition with exact small parts
    f = np.array([1.0, 0.5, 1e-4])
    for p in (0, 1, 7, 10 ** 6, 2 ** 31 - 1, -(2 ** 31)):
        t = orb.turns(np.array([[p, p, p]]), f)
        assert (t >= 0).all() and (t < 2 * math.pi + 1e-12).all()
        for i in range(3):
            # Python's own argument reduction of the exact product is right to the product's rounding
            assert abs(math.remainder(t[0, i] - p * f[i], 2 * math.pi)) <= abs(p * f[i]) * 2.0 ** -52 + 1e-15


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("r", [2, 10, 96, 128])
def test_rotary_oracle_is_complex_multiplication(layout, r):
    g = np.random.default_rng(0)
    x = g.standard_normal((2, 5, 128))
    pos = g.integers(-50, 50, (5, 1))
    f, _ = orb.rotary_freqs(r // 2)
    y = orb.rotary(x, pos, f, layout, [r // 2])
    a = x[..., :r].reshape(2, 5, 2, r // 2).swapaxes(-1, -2) if layout == "half" else x[..., :r].reshape(2, 5, r // 2, 2)
    z = (a[..., 0] + 1j * a[..., 1]) * np.exp(1j * pos * f)
    b = y[..., :r].reshape(2, 5, 2, r // 2).swapaxes(-1, -2) if layout == "half" else y[..., :r].reshape(2, 5, r // 2, 2)
    assert np.abs(b[..., 0] - z.real).max() < 1e-12 and np.abs(b[..., 1] - z.imag).max() < 1e-12
    assert (y[..., r:] == x[..., r:]).all()
    back = orb.rotary(y, pos, f, layout, [r // 2], inverse=True)
    assert np.abs(back - x).max() < 1e-12


def test_rotary_oracle_depends_on_position_differences_only():
    g = np.random.default_rng(1)
    q, k = g.standard_normal((1, 1, 128)), g.standard_normal((1, 1, 128))
    f, _ = orb.rotary_freqs(64)
    dot = lambda p, s: float((orb.rotary(q, np.array([[p]]), f, "half", [64]) * orb.rotary(k, np.array([[s]]), f, "half", [64])).sum())  # noqa: E731
    assert abs(dot(10, 3) - dot(1_000_010, 1_000_003)) < 1e-9


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_gate_norm_oracle_against_torch(pre, post):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, y, gate, scale, shift = r(3, 40), r(3, 40), r(40), r(40), r(40)
    w, b, w2, b2 = r(40), r(40), r(40), r(40)

    def norm(v, kind, w, b):
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, (40,), w, b, 1e-6)
        v = torch.nn.functional.rms_norm(v, (40,), None, 1e-6) if kind == "rms" else v
        return v * w + b
    h = 0.5 * x + 2.0 * gate * norm(y, post, w, b)
    z = norm(h, pre, w2, b2) * (1 + scale) + shift
    n = lambda t: t.numpy()  # noqa: E731
    h2, z2 = orb.gate_norm(n(x), n(y), n(gate), n(scale), n(shift), pre, n(w2), n(b2), post, n(w), n(b), 1e-6, 0.5, 2.0)
    assert np.abs(h2 - n(h)).max() < 1e-12 and np.abs(z2 - n(z)).max() < 1e-11


def test_int8_rows_of_the_oracle():
    g = np.random.default_rng(2)
    x = torch.from_numpy(g.standard_normal((6, 33)).astype(np.float32)).bfloat16().float().numpy()
    x[1] = 0.0
    x[2, 5] = np.inf
    x[3, 0] = np.nan
    x[4] *= 1e-38
    codes, scales = orb.quantize_int8(x)
    assert np.abs(codes).max() == 127
    for m in (0, 5):
        assert np.abs(codes[m] * scales[m].astype(np.float64) - x[m]).max() <= 0.5 * scales[m] * (1 + 2.0 ** -20)
        assert np.abs(codes[m]).max() == 127
    for m in (1, 4):      # below the floor: zero within the floor's step
        assert scales[m] == np.float32(orb.INT8_FLOOR / 127) and not codes[m].any()
    for m in (2, 3):
        assert np.isnan(scales[m]) and not codes[m].any()


def test_linear_oracle_sums_are_whole():
    a = np.full((2, 32768), -127, np.int8)
    w = np.full((3, 32768), 127, np.int8)
    out = orb.linear_int8(a, np.ones(2, np.float32), w, np.ones(3, np.float32))
    assert (out == -127 * 127 * 32768).all() and 127 * 127 * 32768 < 2 ** 31


# ------------------------------------------------------------------ frequencies (host)

@pytest.mark.parametrize("scaling,factor", [("plain", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 8.0), ("by_parts", 2.0)])
@pytest.mark.parametrize("pairs", [1, 2, 21, 64])
def test_frequencies_match_the_oracle(scaling, factor, pairs):
    f, m = bsa.rotary_freqs(pairs, 10000.0, scaling, factor, 4096, device="cpu")
    g, n = orb.rotary_freqs(pairs, 10000.0, scaling, factor, 4096.0)
    assert f.dtype == torch.float64 and np.abs(f.numpy() / g - 1).max() < 1e-13
    assert abs(m - n) <= n * 2.0 ** -24


def test_frequencies_of_several_axes_and_ends():
    f, _ = bsa.rotary_freqs([22, 21, 21], device="cpu")
    assert f.shape == (64,) and f[0] == f[22] == f[43] == 1.0
    f, m = bsa.rotary_freqs(64, 10000.0, "by_parts", 8.0, 4096, device="cpu")
    p, _ = bsa.rotary_freqs(64, device="cpu")
    assert f[0] == p[0] and m == 1.0                           # many turns: kept
    assert abs(f[63] * 8 / p[63] - 1) < 1e-14                  # under one turn: divided
    assert (f <= p).all() and (f >= p / 8).all()


@pytest.mark.parametrize("kw", [dict(pairs=65), dict(pairs=-1), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("inf")),
                                dict(scaling="yarn", factor=2.0, trained_length=0),
                                dict(scaling="yarn", factor=2.0, trained_length=4096, fast_turns=1.0, slow_turns=1.0),
                                dict(scaling="by_parts", factor=2.0, trained_length=4096, slow_turns=-1.0)])
def test_frequency_refusals(kw):
    with pytest.raises(bsa.BsaError) as e:
        bsa.rotary_freqs(**dict(dict(pairs=64, device="cpu"), **kw))
    assert e.value.status == bsa.BSA_ERR_INVALID


# ------------------------------------------------------------------ refusals before any launch

A = 1 << 30       # pretend addresses: never dereferenced, every call below is refused
BIG = 1 << 28


def _rot(ptrs=None, **kw):
    p = dict(B=1, H=4, N=100, D=128, rotary_dim=128, layout=0, axes=1, inverse=0, in_dtype=0, out_dtype=0,
             scale=1.0, eps=1e-6, in_b=100 * 512, in_h=128, in_n=512, out_b=100 * 512, out_h=100 * 128, out_n=128,
             pos_b=0, pos_n=1)
    pairs = kw.pop("axis_pairs", (64,))
    p.update(kw)
    s = bsa.bsa_rotary_params(**p)
    s.axis_pairs = (ctypes.c_int32 * 4)(*pairs)
    a = dict(q=A, k=A + BIG, v=A + 2 * BIG, pos=A, freqs=A, qw=None, kw=None, Q=A + 3 * BIG, K=A + 4 * BIG, V=A + 5 * BIG)
    a.update(ptrs or {})
    return bsa.lib().bsa_rotary(ctypes.byref(s), *[a[n] for n in ("q", "k", "v", "pos", "freqs", "qw", "kw", "Q", "K", "V")], None)


@pytest.mark.parametrize("kw", [dict(D=64), dict(B=0), dict(H=0), dict(N=0), dict(N=(1 << 21) + 1), dict(B=21846),
                                dict(rotary_dim=130, axis_pairs=(65,)), dict(rotary_dim=3), dict(rotary_dim=-2), dict(layout=2),
                                dict(axes=0), dict(axes=5), dict(axis_pairs=(63,)), dict(axes=2, axis_pairs=(65, -1)),
                                dict(in_dtype=2), dict(out_dtype=3), dict(scale=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
                                dict(in_n=-512), dict(out_n=64), dict(out_h=0), dict(pos_n=-1), dict(in_b=1 << 50)])
def test_rotary_invalid_parameters(kw):
    if "in_b" in kw:
        kw = dict(kw, B=2)
    assert _rot(**kw) == bsa.BSA_ERR_INVALID


def test_rotary_pointers():
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    assert bsa.lib().bsa_rotary(None, *[None] * 10, None) == inv
    assert _rot(dict(Q=None)) == inv and _rot(dict(q=None)) == inv
    assert _rot(dict(q=None, k=None, v=None, Q=None, K=None, V=None)) == inv
    assert _rot(dict(pos=None)) == inv and _rot(dict(freqs=None)) == inv
    assert _rot(dict(qw=A), inverse=1) == inv
    assert _rot(dict(q=None, Q=None, qw=A)) == inv                   # a weight without its rows
    assert _rot(dict(Q=A)) == inv                                    # on its input, other strides
    assert _rot(dict(Q=A + 1024)) == inv and _rot(dict(Q=A + BIG)) == inv     # into q, into k
    assert _rot(dict(K=A + 3 * BIG)) == inv                          # two outputs in one place
    assert _rot(dict(q=A + 8)) == al and _rot(dict(V=A + 5 * BIG + 4)) == al
    assert _rot(dict(qw=A + 4)) == al and _rot(dict(freqs=A + 4)) == al and _rot(dict(pos=A + 2)) == al
    assert _rot(in_n=513) == al and _rot(out_n=132, out_h=100 * 132) == al


def _gn(inp=None, h=A + 2 * BIG, z=A + 3 * BIG, zs=None, **kw):
    p = dict(B=2, N=10, C=256, pre=1, post=1, x_dtype=0, y_dtype=0, mod_dtype=1, z_dtype=0, eps=1e-6, residual_scale=1.0,
             branch_scale=1.0)
    for n in "xyhz":
        p[n + "_b"], p[n + "_n"] = 2560, 256
    for n in ("gate", "scale", "shift"):
        p[n + "_b"], p[n + "_n"] = 256, 0
    p.update(kw)
    i = dict(x=A, y=A + BIG, gate=A, scale=A, shift=A)
    i.update(inp or {})
    return bsa.lib().bsa_gate_norm(ctypes.byref(bsa.bsa_gate_norm_params(**p)), ctypes.byref(bsa.bsa_gate_norm_inputs(**i)), h, z, zs, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(N=0), dict(C=0), dict(C=32769), dict(pre=3), dict(post=-1), dict(x_dtype=2),
                                dict(y_dtype=2), dict(mod_dtype=2), dict(z_dtype=3), dict(eps=-1e-6), dict(eps=float("nan")),
                                dict(residual_scale=float("inf")), dict(branch_scale=float("nan")), dict(x_n=-1),
                                dict(h_n=255), dict(z_b=0)])
def test_gate_norm_invalid_parameters(kw):
    assert _gn(**kw) == bsa.BSA_ERR_INVALID


def test_gate_norm_pointers():
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    L = bsa.lib()
    assert L.bsa_gate_norm(None, None, None, None, None, None) == inv
    assert _gn(dict(x=None)) == inv and _gn(h=None, z=None) == inv
    assert _gn(dict(y=None, gate=None)) == inv                       # h without a branch
    assert _gn(dict(y=None), h=None) == inv                          # a gate without a branch
    assert _gn(z=None) == inv                                        # modulation of nothing
    assert _gn(z_dtype=2) == inv and _gn(zs=A) == inv                # codes without scales, scales without codes
    assert _gn(h=A, h_n=512, h_b=5120) == inv                        # on x, other strides
    assert _gn(h=A + 512) == inv and _gn(h=A + BIG) == inv and _gn(z=A) == inv and _gn(z=A + 2 * BIG) == inv
    assert _gn(dict(x=A + 1)) == al and _gn(dict(gate=A + 2)) == al and _gn(dict(pre_bias=A + 2)) == al
    assert _gn(z_dtype=2, zs=A + 1) == al


def _q8(x=A, codes=A + BIG, scale=A, **kw):
    p = dict(B=1, N=10, S=4, L=128, x_dtype=0, x_b=0, x_n=128, x_s=1280, ld=512)
    p.update(kw)
    return bsa.lib().bsa_quantize_int8(ctypes.byref(bsa.bsa_quantize_int8_params(**p)), x, codes, scale, None)


def test_quantize_int8_refusals():
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    for kw in (dict(B=0), dict(N=0), dict(S=0), dict(L=0), dict(S=257), dict(x_dtype=2), dict(ld=511), dict(x_s=-1),
               dict(B=1 << 16, N=1 << 16, x_b=1280)):
        assert _q8(**kw) == inv, kw
    assert _q8(x=None) == inv and _q8(codes=None) == inv and _q8(scale=None) == inv
    assert _q8(codes=A) == inv and _q8(codes=A + 1000) == inv        # over the rows that are read
    assert _q8(x=A + 1) == al and _q8(scale=A + 2) == al


def _lin(a=A, asc=A, w=A + BIG, wsc=A, bias=None, out=A + 2 * BIG, **kw):
    p = dict(M=100, N=200, K=300, out_dtype=0, lda=304, ldw=304, ldo=200)
    p.update(kw)
    return bsa.lib().bsa_linear_int8(ctypes.byref(bsa.bsa_linear_int8_params(**p)), a, asc, w, wsc, bias, out, None)


def test_linear_int8_refusals():
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(K=32769, lda=32784, ldw=32784), dict(out_dtype=2), dict(lda=299), dict(ldw=288),
               dict(ldo=199), dict(lda=-304)):
        assert _lin(**kw) == inv, kw
    for kw in (dict(a=None), dict(asc=None), dict(w=None), dict(wsc=None), dict(out=None), dict(out=A), dict(out=A + BIG + 64)):
        assert _lin(**kw) == inv, kw
    for kw in (dict(a=A + 8), dict(w=A + BIG + 1), dict(lda=301), dict(ldw=312), dict(out=A + 2 * BIG + 1), dict(asc=A + 2), dict(bias=A + 2)):
        assert _lin(**kw) == al, kw


def test_wrappers_refuse_tensors_that_are_not_on_a_device():
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    for call in (lambda: bsa.gate_norm(x), lambda: bsa.quantize_int8(x[0]),
                 lambda: bsa.linear_int8(x[0].to(torch.int8), torch.ones(2), x[0].to(torch.int8), torch.ones(2)),
                 lambda: bsa.rotary(x[:, None], None, None, torch.zeros(2, 1, dtype=torch.int32), torch.ones(64, dtype=torch.float64))):
        with pytest.raises(bsa.BsaError) as e:
            call()
        assert e.value.status == bsa.BSA_ERR_INVALID


def _block(ptr=None, ws=A + 8 * BIG, nbytes=1 << 34, x=A, out=A + BIG, p=None, **kw):
    bp = dict(C=256, x_dtype=0, mod_dtype=1, pre=1, post=1, eps=1e-6, residual_scale=1.0, branch_scale=1.0, qk_eps=1e-6, rope_scale=1.0,
              rotary_dim=128, layout=0, axes=1, gate_b=256, scale_b=256, shift_b=256, pos_n=1, ld_qkv=256, ld_out=256)
    bp.update(kw)
    s = bsa.bsa_block_params(**bp)
    s.axis_pairs = (ctypes.c_int32 * 4)(bp["rotary_dim"] // 2)
    w = dict(gate=A, scale=A, shift=A, w_qkv=A + 2 * BIG, s_qkv=A, w_out=A + 3 * BIG, s_out=A, positions=A, freqs=A)
    w.update(ptr or {})
    p = p or bsa.params(1, 2, 1000, 3)
    return bsa.lib().bsa_forward_block(ctypes.byref(p), ctypes.byref(s), ctypes.byref(bsa.bsa_block_weights(**w)), x, out, ws, nbytes, None)


def test_forward_block_refusals():
    # every step's arguments are checked before the first launch
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    for kw in (dict(C=0), dict(C=32769), dict(x_dtype=2), dict(pre=5), dict(eps=-1.0), dict(rotary_dim=130), dict(qk_eps=float("nan")),
               dict(ld_qkv=128), dict(ld_out=128), dict(nbytes=1000), dict(x=None), dict(out=None), dict(ws=None),
               dict(ws=A), dict(ws=A + BIG - 256), dict(out=A + 256), dict(p=bsa.params(1, 257, 1000, 3)), dict(p=bsa.params(1, 2, 0, 3)),
               dict(ptr=dict(w_qkv=None)), dict(ptr=dict(s_out=None)), dict(ptr=dict(positions=None)), dict(post=-1)):
        assert _block(**kw) == inv, kw
    for kw in (dict(ws=A + 8 * BIG + 16), dict(x=A + 1), dict(ptr=dict(w_out=A + 3 * BIG + 8)), dict(ptr=dict(q_weight=A + 4)),
               dict(ptr=dict(b_out=A + 2)), dict(ld_out=260), dict(ptr=dict(post_bias=A + 1))):
        assert _block(**kw) == al, kw


def test_forward_block_workspace():
    p, bp = bsa.params(1, 56, 37_740, 64), bsa.bsa_block_params(C=7168)
    n = bsa.lib().bsa_forward_block_workspace_bytes(ctypes.byref(p), ctypes.byref(bp))
    rows = 37_740
    want = rows * 7168 + rows * 4 + 3 * rows * 7168 * 2 + bsa.bsa_workspace_bytes(p) + rows * 3 * 7168 * 2
    assert want <= n <= want + 8 * 256
    bp.C = 0
    assert bsa.lib().bsa_forward_block_workspace_bytes(ctypes.byref(p), ctypes.byref(bp)) == 0


def test_linear_int8_refuses_sides_past_32_bit_tiles():
    assert _lin(M=(1 << 30) + 1, K=16, lda=16) == bsa.BSA_ERR_INVALID
    assert _lin(N=2**31 - 1, K=16, ldw=16, ldo=2**31) == bsa.BSA_ERR_INVALID


def test_layout_keys_tell_layouts_apart():
    layout = bsa._load_host().layout
    x = torch.zeros(4, 6, 8)
    same = torch.ones(4, 6, 8)
    assert layout(x, None) == layout(same, None)                    # never the address or the values
    others = [(x,), (None, x), (x, x), (x.bfloat16(), None), (x.int(), None), (x.transpose(0, 1), None), (x[:2], None), (x[..., :4], None),
              (x.reshape(24, 8), None), (x[0], None), (x[:, :1].expand(4, 6, 8), None), (x.to("meta"), None)]
    keys = [layout(*t) for t in others] + [layout(x, None)]
    assert len(set(keys)) == len(keys)
    with pytest.raises(TypeError):
        layout(x, 3)


def test_host_outputs_and_calls_check_their_arguments():
    host, x = bsa._load_host(), torch.zeros(3)
    y = host.empty((2, 5), (16, 1), torch.int8, x)
    assert y.shape == (2, 5) and y.stride() == (16, 1) and y.dtype is torch.int8 and y.device == x.device
    for bad in (lambda: host.empty((2,), (1, 1), torch.int8, x), lambda: host.empty((-1,), (1,), torch.int8, x),
                lambda: host.empty((1,), (1,), "int8", x), lambda: host.empty((1,) * 9, (1,) * 9, torch.int8, x),
                lambda: host.call(), lambda: host.call(0), lambda: host.call(1, "x"), lambda: host.call(1, *range(13)),
                lambda: host.call(1, (None,) * 17)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            bad()
    at = bsa.lib().addresses
    assert host.call(at["bsa_quantize_int8"], None, x, x, x, None) == bsa.BSA_ERR_INVALID
    assert host.call(at["bsa_gate_norm"], None, (x, None), x, None, None, None) == bsa.BSA_ERR_INVALID


@pytest.fixture
def launches(monkeypatch):
    """The wrappers on CPU tensors with the library call replaced: what each call would have passed."""
    real, seen = bsa._load_host(), []

    class Host:
        layout, empty = staticmethod(real.layout), staticmethod(real.empty)

        @staticmethod
        def call(at, params, *args):
            name = next(n for n, a in bsa.lib().addresses.items() if a == at)
            kind = bsa._SIGS[name][1][0]._type_
            seen.append((name, kind.from_buffer_copy(ctypes.string_at(params, ctypes.sizeof(kind))), args))
            return 0
    monkeypatch.setattr(bsa, "_host", Host)
    monkeypatch.setattr(bsa, "_one_device", lambda *a: 0)
    monkeypatch.setattr(bsa, "_device_now", lambda: 0)
    monkeypatch.setattr(bsa, "_raw_stream", lambda device: 0)
    return seen


def test_scalars_are_read_at_every_call(launches):
    # numbers held in tensors of no dimension (a learned layer scale), changed in place between two calls
    x = torch.zeros(1, 2, 128)
    s = {n: torch.tensor(0.5) for n in ("eps", "residual_scale", "branch_scale")}
    q, pos, freqs = torch.zeros(1, 2, 3, 128), torch.zeros(3, dtype=torch.int32), torch.ones(64, dtype=torch.float64)
    m, inverse, pairs = torch.tensor(0.5), torch.tensor(False), torch.tensor([64])
    for value in (0.5, 2.0):
        for t in s.values():
            t.fill_(value)
        bsa.gate_norm(x, x, **s)
        p = launches[-1][1]
        assert (p.eps, p.residual_scale, p.branch_scale) == (value,) * 3
        m.fill_(value)
        inverse.fill_(value > 1)
        bsa.rotary(q, None, None, pos, freqs, scale=m, eps=m, inverse=inverse, axis_pairs=pairs)
        p = launches[-1][1]
        assert (p.scale, p.eps, p.inverse, p.axis_pairs[0]) == (value, value, int(value > 1), 64)
    want_z = torch.tensor(True)
    assert bsa.gate_norm(x, x, want_z=want_z)[1] is not None
    want_z.fill_(False)
    assert bsa.gate_norm(x, x, want_z=want_z)[1] is None and launches[-1][2][2] is None


# A call that passes every check goes on to the device; without one it reports BSA_ERR_CUDA there.
checks_alone = pytest.mark.skipif(torch.cuda.is_available(), reason="pretend addresses would be launched on")


def _packed(**kw):
    """Views of one buffer of rows [N, groups, H, 128], in and out."""
    return dict(dict(in_b=0, in_h=128, in_n=7 * 512, out_b=0, out_h=128, out_n=7 * 512), **kw)


def test_rotary_in_place_refuses_rows_that_another_tensor_reads():
    inv, step = bsa.BSA_ERR_INVALID, 1024          # bytes of a group's rows of 4 heads
    q, k, v, K, V = A, A + step, A + 2 * step, A + 4 * BIG, A + 5 * BIG
    at = lambda **p: _rot(dict(dict(q=q, k=k, v=v, Q=q, K=k, V=v), **p), **_packed())  # noqa: E731
    assert at(k=q, K=K) == inv          # one input twice, turned in place once
    assert at(v=k, V=V) == inv          # k and v tied
    assert at(k=q + 256, K=K) == inv    # k starts at q's second head
    assert at(v=q + 7 * step, V=V) == inv        # at q's second token
    assert at(v=q + 7 * step * 98 + 768, V=V) == inv
    assert at(V=k) == inv and at(K=K, V=K + 768) == inv


def test_rotary_outputs_do_not_overlap():
    inv, Q = bsa.BSA_ERR_INVALID, A + 3 * BIG
    for off in (256, 1024, 100 * 256, 3 * 100 * 256, 4 * 100 * 256 - 256):
        assert _rot(dict(K=Q + off)) == inv and _rot(dict(V=Q + off)) == inv
        assert _rot(dict(K=Q - off)) == inv


@checks_alone
def test_rotary_takes_rows_that_interleave():
    ok, step = bsa.BSA_ERR_CUDA, 1024
    at = lambda **p: _rot(dict(dict(q=A, k=A + step, v=A + 2 * step), **p), **_packed())  # noqa: E731
    assert at(Q=A, K=A + step, V=A + 2 * step) == ok                               # in place
    assert at(Q=A + 3 * step, K=A + 4 * step, V=A + 5 * step) == ok                # beside its inputs
    assert at(k=A, v=A, Q=A + 3 * step, K=A + 4 * step, V=A + 5 * step) == ok      # one input read three times
    assert _rot(dict(K=A + 3 * BIG + 4 * 100 * 256)) == ok                         # Q and K one after the other


@checks_alone
def test_rotary_overlap_check_against_every_row():
    # in place q, k at any offset with the same strides: refused exactly where two rows share a byte
    g, met = np.random.default_rng(3), 0
    for _ in range(400):
        n = [int(g.integers(1, 4)) for _ in range(3)]
        order, s, reach = g.permutation(3), [0, 0, 0], 128
        for i in order:
            s[i] = reach + 8 * int(g.integers(0, 40))
            reach += (n[i] - 1) * s[i]
        rows = np.array([2 * (b * s[0] + h * s[1] + t * s[2]) for b in range(n[0]) for h in range(n[1]) for t in range(n[2])])
        off = 16 * int(g.integers(-reach // 8 - 2, reach // 8 + 3))
        want = bool((np.abs(rows[:, None] - rows[None] - off) < 256).any())
        st = dict(in_b=s[0], in_h=s[1], in_n=s[2], out_b=s[0], out_h=s[1], out_n=s[2])
        got = _rot(dict(q=A, Q=A, k=A + off, K=A + 4 * BIG, v=None, V=None), B=n[0], H=n[1], N=n[2], **st)
        assert got == (bsa.BSA_ERR_INVALID if want else bsa.BSA_ERR_CUDA), (n, s, off)
        met += want
    assert 0 < met < 400      # both kinds were drawn


@pytest.mark.parametrize("name", ["gate", "scale", "shift", "pre_weight", "pre_bias", "post_weight", "post_bias"])
def test_gate_norm_outputs_over_a_vector(name):
    inv, h, z = bsa.BSA_ERR_INVALID, A + 2 * BIG, A + 3 * BIG
    per = dict(gate_b=2560, gate_n=256, scale_b=2560, scale_n=256, shift_b=2560, shift_n=256)
    for out in (h, z):
        for kw in ({}, per):                                     # one vector a batch entry, one a token
            assert _gn({name: out}, **kw) == inv
            assert _gn({name: out + 2 * 19 * 256}, **kw) == inv      # from the last row on
    if name in ("gate", "scale", "shift"):
        assert _gn({name: h}, mod_dtype=0, **per) == inv             # of the rows' own type and strides
        assert _gn({name: z - 4 * 5000}, **per) == inv               # ends inside z


@checks_alone
def test_gate_norm_takes_rows_that_interleave():
    wide = dict({n + "_b": 8 * 2560 for n in "xyhz"}, **{n + "_n": 8 * 256 for n in "xyhz"})
    mods = {f"{n}_{d}": 8 * (2560 if d == "b" else 256) for n in ("gate", "scale", "shift") for d in "bn"}
    part = [A + 512 * i for i in range(8)]
    inp = dict(x=part[0], y=part[1], gate=part[2], scale=part[3], shift=part[4])
    for h in (part[5], part[0]):                                     # beside the inputs, or in place
        assert _gn(inp, h=h, z=part[6], mod_dtype=0, **wide, **mods) == bsa.BSA_ERR_CUDA
    assert _gn(inp, h=part[5], z=part[5], mod_dtype=0, **wide, **mods) == bsa.BSA_ERR_INVALID
    assert _gn(inp, h=part[5], z=part[5] + 256, mod_dtype=0, **wide, **mods) == bsa.BSA_ERR_INVALID


@pytest.mark.parametrize("name", ["gate", "scale", "shift", "w_qkv", "s_qkv", "b_qkv", "w_out", "s_out", "b_out", "pre_weight", "pre_bias",
                                  "post_weight", "post_bias", "q_weight", "k_weight", "positions", "freqs"])
def test_forward_block_workspace_and_result_lie_apart_from_what_is_read(name):
    inv, ws = bsa.BSA_ERR_INVALID, A + 8 * BIG
    p, bp = bsa.params(1, 2, 1000, 3), bsa.bsa_block_params(C=256)
    n = bsa.lib().bsa_forward_block_workspace_bytes(ctypes.byref(p), ctypes.byref(bp))
    for at in (ws, ws + n // 2 // 256 * 256, ws + n - 256, A + BIG, A + BIG + 512 * 999):
        assert _block(ptr={name: at}) == inv, hex(at)
    for bases in (dict(), {name: ws + n}):
        if not torch.cuda.is_available():
            assert _block(ptr=bases) == bsa.BSA_ERR_CUDA        # every check passed


def _rot_each(ptrs=None, own=None, **kw):
    """q with 4 heads, k and v with 2, each in an allocation of its own."""
    base = dict(B=1, H=4, N=100, D=128, rotary_dim=128, layout=0, axes=1, inverse=0, in_dtype=0, out_dtype=0, scale=1.0, eps=1e-6,
                in_b=0, in_h=128, in_n=512, out_b=0, out_h=100 * 128, out_n=128, pos_b=0, pos_n=1)
    s = (bsa.bsa_rotary_params * 3)()
    for i, n in enumerate("qkv"):
        p = dict(base, **kw)
        if i:
            p.update(H=2, in_n=256)
        p.update((own or {}).get(n, {}))
        s[i] = bsa.bsa_rotary_params(**p)
        s[i].axis_pairs = (ctypes.c_int32 * 4)(64)
    a = dict(q=A, k=A + BIG, v=A + 2 * BIG, pos=A, freqs=A, qw=None, kw=None, Q=A + 3 * BIG, K=A + 4 * BIG, V=A + 5 * BIG)
    a.update(ptrs or {})
    return bsa.lib().bsa_rotary_each(s, *[a[n] for n in ("q", "k", "v", "pos", "freqs", "qw", "kw", "Q", "K", "V")], None)


def test_rotary_each_refusals():
    inv, al = bsa.BSA_ERR_INVALID, bsa.BSA_ERR_ALIGN
    assert bsa.lib().bsa_rotary_each(None, *[None] * 10, None) == inv
    assert _rot_each(dict(q=None, k=None, v=None, Q=None, K=None, V=None)) == inv
    assert _rot_each(dict(q=None, Q=None, qw=A)) == inv and _rot_each(dict(V=None)) == inv and _rot_each(dict(pos=None)) == inv
    # what one tensor alone would be refused for, in any place
    for n in "qkv":
        for bad in (dict(H=0), dict(in_n=-1), dict(out_n=64), dict(in_dtype=2), dict(in_b=1 << 50, B=2)):
            assert _rot_each(own={n: bad}) == inv, (n, bad)
        assert _rot_each({n: A + BIG * "qkv".index(n) + 8}) == al and _rot_each({n.upper(): A + BIG * (3 + "qkv".index(n)) + 8}) == al
        assert _rot_each(own={n: dict(in_n=516)}) == al
    # parameters of the turn that differ
    for bad in (dict(N=99), dict(B=2), dict(rotary_dim=126), dict(layout=1), dict(inverse=1), dict(scale=2.0), dict(eps=0.0), dict(pos_n=2)):
        assert _rot_each(own=dict(v=bad)) == inv, bad
    # outputs over the rows of a tensor that another launch reads or writes
    inplace = dict(q=dict(out_h=128, out_n=512))
    assert _rot_each(dict(Q=A, k=A + 1024, K=A + 4 * BIG), own=inplace) == inv
    assert _rot_each(dict(Q=A + BIG)) == inv and _rot_each(dict(K=A)) == inv and _rot_each(dict(V=A + 3 * BIG + 4 * 100 * 256 - 256)) == inv
    assert _rot_each(dict(K=A + 5 * BIG + 256)) == inv


@checks_alone
def test_rotary_each_passes_what_lies_apart():
    cu = bsa.BSA_ERR_CUDA
    inplace = dict(q=dict(out_h=128, out_n=512), k=dict(out_h=128, out_n=256), v=dict(out_h=128, out_n=256))
    assert _rot_each() == cu and _rot_each(dict(qw=A, kw=A)) == cu
    assert _rot_each(dict(Q=A, K=A + BIG, V=A + 2 * BIG), own=inplace) == cu
    assert _rot_each(dict(v=A + BIG)) == cu and _rot_each(own=dict(k=dict(pos_b=5))) == cu
    assert _rot_each(dict(q=None, Q=None)) == cu and _rot_each(own=dict(q=dict(in_dtype=1, in_n=640))) == cu


def test_rotary_of_several_layouts_is_one_call(launches):
    # nothing runs before all of it was checked, an output over another tensor's rows among that
    pos, freqs = torch.zeros(3, dtype=torch.int32), torch.ones(64, dtype=torch.float64)
    q, k, v = torch.zeros(1, 4, 3, 128), torch.zeros(1, 2, 3, 128), torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    Q, K, V = bsa.rotary(q, k, v, pos, freqs, q_weight=torch.ones(128))
    assert Q.shape == q.shape and K.shape == k.shape and V.dtype == v.dtype
    assert len(launches) == 1 and launches[0][0] in ("bsa_rotary", "bsa_rotary_each")
    assert [a is not None for a in launches[0][2]] == [True] * 6 + [False] + [True] * 4
    bsa.rotary(q, k, None, pos, freqs)
    bsa.rotary(q, q.clone(), q.clone(), pos, freqs)
    assert len(launches) == 3


def test_warps_of_the_product_wait_as_one():
    # a wait that runs out is answered lane by lane; barriers that count a warp follow, so all its lanes have to go on or none
    text = open(os.path.join(os.path.dirname(bsa.__file__), "csrc", "linear_int8.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    for kernel in re.split(r"__global__", text)[1:]:
        # the warps that read accumulators: after the producer's and the issuer's branches
        warps = kernel[kernel.index("} else if (warp < "):]
        assert re.findall(r"mbar_wait\w*\(&ctl->(\w+)", warps) == ["acc_full"] and "mbar_wait_warp(&ctl->acc_full" in warps
    # sums are used only where no CTA of the cluster gave up
    few = text[text.index("linear_int8_few_kernel("):text.index("int few_split")]
    assert few.index("map_to_rank(&ctl->abort_flag") < few.index("a.w_scale")
    # and multiplications that were issued are waited for before their accumulators are freed
    for kernel in re.split(r"__global__", text)[1:]:
        assert kernel.index("&ctl->fin, 0, wc") < kernel.index("tmem_dealloc")


@pytest.mark.parametrize("name", ["rotary.cu", "gate_norm.cu", "quant_int8.cu", "linear_int8.cu", "rows.cuh"])
def test_kernels_that_start_early_read_through_the_coherent_path(name):
    # A kernel that is resident while the one before it still writes may not use read-only loads: they hold for memory that
    # nobody writes during the kernel's life, and nothing orders them after the wait.
    text = open(os.path.join(os.path.dirname(bsa.__file__), "csrc", name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    for word in ("__ldg", "ld.global.nc", "ld_stream_v4", "__ldcs", "__restrict__"):
        assert word not in text, word
    if name.endswith(".cu"):
        assert text.count("__global__") == text.count("grid_wait();") == text.count("grid_ready();")


def test_host_module_is_tied_to_its_torch_and_python(monkeypatch, tmp_path):
    from block_sparse_video_bsa_b200 import build
    module = bsa._load_host()
    assert module.built_for == build.host_built_for() and torch.__version__ in module.built_for
    source, made, stamp = (str(tmp_path / n) for n in ("host.cpp", "host.so", "stamp"))
    monkeypatch.setattr(build, "HOST", made)
    monkeypatch.setattr(build, "HOST_STAMP", stamp)
    for path, text in ((source, ""), (made, ""), (stamp, module.built_for)):
        assert not build._host_current(source)
        with open(path, "w") as f:
            f.write(text)
    assert build._host_current(source)
    monkeypatch.setattr(build, "host_built_for", lambda: "torch 0.0, Python 0.0")
    assert not build._host_current(source)                                   # built again
    monkeypatch.setattr(bsa, "_host", None)
    with pytest.raises(RuntimeError, match="torch 0.0, Python 0.0"):         # and not used before that
        bsa._load_host()


def test_wrappers_have_a_device_and_a_stream_on_every_torch():
    # under a torch without the private accessors
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    hasattr(torch._C, n) and delattr(torch._C, n)\n"
            "from block_sparse_video_bsa_b200 import bsa\n"
            "assert callable(bsa._device_now) and callable(bsa._raw_stream)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(bsa.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_host_calls_get_a_tensor_of_its_own():
    # a lazy clone shares its source's memory until it is written: an output's address has to be its own
    if not hasattr(torch.Tensor, "_lazy_clone"):
        pytest.skip("this torch has no lazy clones")
    seen = []
    record = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 5)(lambda *a: seen.extend(a) or 0)
    x = torch.zeros(64)
    y = x._lazy_clone()
    assert bsa._load_host().call(ctypes.cast(record, ctypes.c_void_p).value, y, None, None, None, None) == 0
    assert seen[0] == y.data_ptr() != x.data_ptr() and seen[1:] == [None] * 4


def test_rotary_weights_of_absent_tensors_are_not_looked_at(launches):
    pos, freqs, w = torch.zeros(3, dtype=torch.int32), torch.ones(64, dtype=torch.float64), torch.ones(128)
    q, k = torch.zeros(1, 4, 3, 128), torch.zeros(1, 2, 3, 128)
    for given in ((q, None, None), (None, k, None), (None, None, k), (q, None, k), (None, k, q)):
        bsa.rotary(*given, pos, freqs, q_weight=w, k_weight=w)
        args = launches[-1][2]
        assert [a is not None for a in args[:3]] == [t is not None for t in given]
        assert [a is not None for a in args[5:7]] == [t is not None for t in given[:2]]


@checks_alone
def test_rotary_overlap_check_of_other_head_counts_and_types():
    # as above with rows of several layouts: k has heads of its own, and rows of 256 or 512 bytes
    g, met = np.random.default_rng(4), 0
    for _ in range(600):
        wide = int(g.integers(0, 2))
        n = [int(g.integers(1, 4)) for _ in range(3)]
        heads = int(g.integers(1, 5))
        order, s, reach = g.permutation(3), [0, 0, 0], 256
        for i in order:
            s[i] = reach + 16 * int(g.integers(0, 60))
            reach += (max(n[i], heads if i == 1 else 0) - 1) * s[i]
        starts = lambda h: np.array([2 * (b * s[0] + i * s[1] + t * s[2]) for b in range(n[0]) for i in range(h) for t in range(n[2])])  # noqa: E731
        off = 16 * int(g.integers(-reach // 8 - 2, reach // 8 + 3))
        d = starts(heads)[:, None] + off - starts(n[1])[None]
        want = bool(((d < 256) & (-d < 256 * (1 + wide))).any())
        st = dict(in_b=s[0], in_h=s[1], in_n=s[2], out_b=s[0], out_h=s[1], out_n=s[2])
        half = [x // 2 for x in s] if wide else s
        k = dict(H=heads, in_dtype=wide, in_b=half[0], in_h=half[1], in_n=half[2], out_b=s[0], out_h=s[1], out_n=s[2])
        got = _rot_each(dict(q=A, Q=A, k=A + off, K=A + 4 * BIG, v=None, V=None), own=dict(q=dict(H=n[1]), k=k), B=n[0], N=n[2], **st)
        assert got == (bsa.BSA_ERR_INVALID if want else bsa.BSA_ERR_CUDA), (n, heads, s, off, wide)
        met += want
    assert 0 < met < 600


@checks_alone
def test_gate_norm_takes_vectors_beside_its_rows():
    # [B, 1 + N, C]: the first row of an entry is its gate, the rest are its rows, updated in place; and one vector before all rows
    rows = dict({n + "_b": 11 * 256 for n in "xh"}, x_n=256, h_n=256, scale_b=0, shift_b=0)
    assert _gn(dict(x=A + 512, gate=A, scale=A, shift=A), h=A + 512, mod_dtype=0, gate_b=11 * 256, **rows) == bsa.BSA_ERR_CUDA
    assert _gn(dict(x=A + 512, gate=A), h=A + 512, mod_dtype=0, gate_b=0, **rows) == bsa.BSA_ERR_CUDA
    assert _gn(dict(x=A + 512, gate=A + 2), h=A + 512, mod_dtype=0, gate_b=11 * 256, **rows) == bsa.BSA_ERR_INVALID
    assert _gn(dict(x=A + 512, gate=A), h=A + 512, mod_dtype=0, gate_b=12 * 256, **rows) == bsa.BSA_ERR_INVALID


@checks_alone
def test_forward_block_workspace_between_rows_that_are_read():
    # one arena: an entry's gate, then the workspace, then the next entry's gate
    p, bp = bsa.params(2, 2, 1000, 3), bsa.bsa_block_params(C=256)
    n = bsa.lib().bsa_forward_block_workspace_bytes(ctypes.byref(p), ctypes.byref(bp))
    ws = A + 8 * BIG
    for gap in (1024, 1020, 256):                                # the gate's 256 values fit in the first gap alone
        gate_b = (gap + n) // 4 + 256
        rc = _block(ptr=dict(gate=ws - gap), gate_b=gate_b, p=p, ws=ws)
        assert rc == (bsa.BSA_ERR_CUDA if gap == 1024 else bsa.BSA_ERR_INVALID)
