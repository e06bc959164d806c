"""Cases of the operators around the block-sparse attention: rotary positions (with the per-head norm and the
head-major layout the attention reads), the gated and modulated norms at a block's ends, and the int8
projections with a scale for each token and channel.

Each case is one call as a program around the attention makes it; the plain form beside it is written from the
formulas in elementary torch operations.
"""

import math

import torch

own = False

HEAD = 128            # head dimension of the attention
FLOOR = 2.0 ** -100   # smallest row maximum the int8 scale is taken from


# ------------------------------------------------------------------ cases

def _rotary(name, B, H, N, r, layout, axes, norm, dtype="bf16", scaling="none", factor=1.0, start=0,
            inverse=False, tensors=3):
    c = dict(op="rotary", B=B, H=H, N=N, r=r, layout=layout, axes=axes, norm=norm, dtype=dtype,
             scaling=scaling, factor=float(factor), start=start, inverse=inverse, tensors=tensors)
    return dict(c, name=name) if name else c


def _norm(name, B, N, C, pre, post, stream="bf16", mod="batch", mod_dtype="fp32", branch=True,
          affine=True):
    c = dict(op="norm", B=B, N=N, C=C, pre=pre, post=post, stream=stream, mod=mod,
             mod_dtype=mod_dtype, branch=branch, affine=affine)
    return dict(c, name=name) if name else c


def _linear(name, M, K, N, bias=True, out="bf16", norm=False, heads=0):
    c = dict(op="linear", M=M, K=K, N=N, bias=bias, out=out, norm=norm, heads=heads)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of a stream, 56 heads: its q, k and v after the projection, far into the sequence
        _rotary("rotary-1-token", 1, 56, 1, 128, "half", 1, True, scaling="yarn", factor=8, start=1_000_000),
        # a small layer of 2 heads and 2,048 tokens: half the head rotated, q and k only, fp32 rows
        _rotary("rotary-2k-2-heads", 1, 2, 2_048, 64, "interleaved", 1, False, dtype="fp32",
                scaling="linear", factor=4, tensors=2),
        # 768p, 5 s of video: t, h, w positions, q and k normed, token-major projection to head-major Q, K, V
        _rotary("rotary-768p-5s", 1, 56, 37_740, 128, "interleaved", 3, True),
        # 2K, 5 s of video: the longest sequence; 96 of 128 dimensions, halves layout
        _rotary("rotary-2K-5s", 1, 56, 133_644, 96, "half", 3, True, scaling="ntk", factor=4),
        # one row: the modulated norm of a single token
        _norm("norm-1-row", 1, 1, 7_168, "rms", "rms"),
        # a batch of short text sequences of odd width, fp32 residual, one modulation vector a token
        _norm("norm-text-fp32", 3, 515, 1_111, "layer", "none", stream="fp32", mod="token", mod_dtype="bf16"),
        # 768p, 5 s: end of the attention branch (norm, gate, residual) and start of the next (norm, modulation)
        _norm("norm-768p-5s", 1, 37_740, 7_168, "layer", "rms", affine=False),
        # 768p, 15 s, fp32 residual stream and bf16 modulation
        _norm("norm-768p-15s-fp32", 1, 103_996, 7_168, "rms", "none", stream="fp32", mod_dtype="bf16"),
        # one token through the output projection
        _linear("linear-1-token", 1, 7_168, 7_168),
        # a 512-token text prefix from the modulated norm into the QKV projection
        _linear("linear-norm-512", 512, 7_168, 21_504, norm=True),
        # an odd small layer
        _linear("linear-odd", 1_000, 1_111, 515, out="fp32"),
        # 768p, 5 s: the attention's head-major output through the output projection
        _linear("linear-768p-5s", 37_740, 7_168, 7_168, heads=56),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "norm", "linear"))
    if op == "rotary":
        B, H = rng.choice((1, 1, 2, 3)), rng.choice((1, 2, 5, 12, 40, 56))
        most = 133_644 * 56 // (B * H)
        dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
        N = _log(rng, 1, min(133_644, most // (2 if dtype == "fp32" else 1)))
        r = rng.choice((128, 128, 64, 96, 32, 2 * rng.randrange(3, 65)))
        scaling = rng.choice(("none", "linear", "ntk", "yarn"))
        inverse = rng.random() < 0.2
        return _rotary(None, B, H, N, r, rng.choice(("half", "interleaved")), rng.choice((1, 3)),
                       (not inverse) and rng.random() < 0.6, dtype, scaling,
                       1.0 if scaling == "none" else rng.choice((2, 4, 8)),
                       rng.choice((0, 0, rng.randrange(1, 2_000_000))), inverse, rng.choice((1, 2, 3)))
    if op == "norm":
        B = rng.choice((1, 1, 2, 3))
        C = rng.choice((7_168, 5_120, 256, 8 * _log(rng, 8, 1_536), _log(rng, 64, 12_288)))
        stream, mod = rng.choice(("bf16", "bf16", "fp32")), rng.choice(("batch", "batch", "token", "none"))
        most = 37_740 * 7_168 // (B * C)
        N = _log(rng, 1, max(2, min(60_000, most)))
        return _norm(None, B, N, C, rng.choice(("rms", "layer", "none")), rng.choice(("rms", "layer", "none")),
                     stream, mod, rng.choice(("fp32", "bf16")), rng.random() < 0.8, rng.random() < 0.5)
    heads = rng.choice((0, 0, 0, 2, 40, 56))
    K = heads * HEAD if heads else rng.choice((7_168, 256, 16 * _log(rng, 4, 1_792), _log(rng, 64, 16_384)))
    N = rng.choice((7_168, 21_504, 8 * _log(rng, 2, 2_688), _log(rng, 16, 16_384)))
    most = 37_740 * 7_168 * 7_168 // (K * N)
    M = _log(rng, 1, max(2, min(40_000, most)))
    return _linear(None, M, K, N, rng.random() < 0.6, rng.choice(("bf16", "bf16", "fp32")),
                   not heads and K <= 16_384 and rng.random() < 0.3, heads)


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _pairs(r, axes):
    """Pairs of each axis: all for one, or t, h, w with the odd ones to t."""
    n = r // 2
    return [n] if axes == 1 else [n - 2 * (n // 3), n // 3, n // 3]


def _freqs(c):
    """Radians a position of every pair (64 bits) and the factor on cos and sin, as the model's config gives them."""
    out, m, base, f = [], 1.0, 10_000.0, c["factor"]
    if c["scaling"] == "yarn":
        m = 0.1 * math.log(f) + 1.0
    for n in _pairs(c["r"], c["axes"]):
        b = base * f ** (n / (n - 1)) if c["scaling"] == "ntk" and n > 1 else base
        for i in range(n):
            w = b ** (-i / n)
            if c["scaling"] == "linear":
                w /= f
            elif c["scaling"] == "yarn":
                turns = 4_096 * w / (2 * math.pi)   # over the trained length
                keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
                w = w * keep + w / f * (1.0 - keep)
            out.append(w)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), m


def _positions(c):
    """[N, axes] int32: one running index, or the t, h, w of a raster of 24 x 40 patches a frame."""
    t = torch.arange(c["N"], device="cuda") + c["start"]
    if c["axes"] == 1:
        return t[:, None].to(torch.int32).contiguous()
    return torch.stack((t // 960, t // 40 % 24, t % 40), 1).to(torch.int32).contiguous()


def _prepare_rotary(c, g):
    B, H, N, n = c["B"], c["H"], c["N"], c["tensors"]
    dt = _TYPES[c["dtype"]]
    if c["inverse"]:      # rows of the attention's own layout, back to the model's axes
        x = _randn(g, n, B, H, N, HEAD, dtype=dt)
        parts = [x[i] for i in range(n)]
    else:                 # one projection's token-major rows
        x = _randn(g, B, N, n, H, HEAD, dtype=dt)
        parts = [x[:, :, i].transpose(1, 2) for i in range(n)]
    freqs, m = _freqs(c)
    pairs = _pairs(c["r"], c["axes"])
    axis = torch.tensor([a for a, k in enumerate(pairs) for _ in range(k)], device="cuda")
    s = dict(c=c, parts=parts, freqs=freqs, m=m, positions=_positions(c), pairs=pairs, axis=axis, weights=[None, None])
    if c["norm"]:
        s["weights"] = [1.0 + 0.1 * _randn(g, HEAD) for _ in range(2)]
    return s


def _prepare_norm(c, g):
    B, N, C = c["B"], c["N"], c["C"]
    loud = 1.0 + 9.0 * (torch.rand(C, generator=g, device="cuda") < 0.01)    # a few large channels, as in a trained stream
    s = dict(c=c, x=(_randn(g, B, N, C) * loud).to(_TYPES[c["stream"]]), y=None, gate=None, scale=None, shift=None)
    if c["branch"]:
        s["y"] = _randn(g, B, N, C, dtype=torch.bfloat16)
    if c["mod"] != "none":
        shape = (B, 1, C) if c["mod"] == "batch" else (B, N, C)
        s["scale"], s["shift"] = ((0.3 * _randn(g, *shape)).to(_TYPES[c["mod_dtype"]]) for _ in range(2))
        if c["branch"]:
            s["gate"] = (0.5 * _randn(g, *shape)).to(_TYPES[c["mod_dtype"]])
    for k in ("pre", "post"):
        on = c["affine"] and c[k] != "none"
        s[k + "_weight"] = 1.0 + 0.1 * _randn(g, C) if on else None
        s[k + "_bias"] = 0.1 * _randn(g, C) if on and c[k] == "layer" else None
    return s


def _prepare_linear(c, g):
    M, K, N = c["M"], c["K"], c["N"]
    s = dict(c=c, bias=0.1 * _randn(g, N) if c["bias"] else None)
    if c["heads"]:        # attention output, head-major
        s["x"] = _randn(g, 1, c["heads"], M, HEAD, dtype=torch.bfloat16)
    else:
        loud = 1.0 + 9.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, M, K) * loud).to(torch.bfloat16)
    if c["norm"]:
        s["scale"], s["shift"] = (0.3 * _randn(g, 1, 1, K) for _ in range(2))
    w = _randn(g, N, K)
    top = w.abs().amax(1, keepdim=True)
    w.mul_(127.0 / top).round_()
    # rows of the stored weight start on 16 bytes, as a program lays it out once
    s["w8"] = torch.zeros(N, -(-K // 16) * 16, dtype=torch.int8, device="cuda")[:, :K]
    s["w8"].copy_(w)
    s["w_scale"] = (top[:, 0] / (127.0 * math.sqrt(K))).contiguous()
    return s


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "norm": _prepare_norm, "linear": _prepare_linear}[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------ plain forms

def _plain_rotary(s):
    c, h = s["c"], s["c"]["r"] // 2
    angle = s["positions"].double()[:, s["axis"]] * s["freqs"]             # [N, r/2]: far positions need 64 bits
    cos, sin = (angle.cos() * s["m"]).float(), (angle.sin() * s["m"]).float()
    if c["inverse"]:
        sin = -sin
    out = []
    for i, x in enumerate(s["parts"]):
        x = x.float()
        if i == 2:                                                    # v: the layout alone
            out.append(x.to(_TYPES[c["dtype"]]).contiguous())
            continue
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weights"][i]
        if c["layout"] == "half":
            a, b = x[..., :h], x[..., h:2 * h]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        out.append(torch.cat((turned, x[..., 2 * h:]), -1).to(_TYPES[c["dtype"]]).contiguous())
    return out


def _plain_normed(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    if kind != "none":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        x = x * weight
    return x if bias is None else x + bias


def _plain_norm(s):
    c, h = s["c"], s["x"].float()
    if s["y"] is not None:
        y = _plain_normed(s["y"].float(), c["post"], s["post_weight"], s["post_bias"])
        h = h + (y if s["gate"] is None else y * s["gate"].float())
    z = _plain_normed(h, c["pre"], s["pre_weight"], s["pre_bias"])
    if s["scale"] is not None:
        z = z * (1.0 + s["scale"].float()) + s["shift"].float()
    return {"h": h.to(_TYPES[c["stream"]]) if s["y"] is not None else None, "z": z.to(torch.bfloat16)}


def _plain_linear(s):
    c, x = s["c"], s["x"].float()
    if c["heads"]:
        x = x[0].transpose(0, 1).reshape(c["M"], c["K"])
    if c["norm"]:
        x = _plain_normed(x, "rms", None, None) * (1.0 + s["scale"][0]) + s["shift"][0]
    top = x.abs().amax(1, keepdim=True).clamp(min=FLOOR)
    most = torch.full_like(top, 127.0)
    codes = (x * (most / top)).round()
    out = (codes @ s["w8"].float().t()) * (top / most) * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(_TYPES[c["out"]])


# ------------------------------------------------------------------ the framework's calls

def _own_rotary(s):
    from block_sparse_video_bsa_b200 import bsa
    c, p = s["c"], s["parts"] + [None] * (3 - len(s["parts"]))
    out = bsa.rotary(p[0], p[1], p[2], s["positions"], s["freqs"], layout=c["layout"], axis_pairs=s["pairs"], q_weight=s["weights"][0],
                     k_weight=s["weights"][1] if p[1] is not None else None, eps=1e-6, scale=s["m"], inverse=c["inverse"])
    return list(out[:c["tensors"]])


def _own_norm(s):
    from block_sparse_video_bsa_b200 import bsa
    c = s["c"]
    h, z = bsa.gate_norm(s["x"], s["y"], gate=s["gate"], scale=s["scale"], shift=s["shift"], pre=c["pre"], pre_weight=s["pre_weight"],
                         pre_bias=s["pre_bias"], post=c["post"], post_weight=s["post_weight"], post_bias=s["post_bias"], eps=1e-6)
    return {"h": h if s["y"] is not None else None, "z": z}


def _own_linear(s):
    from block_sparse_video_bsa_b200 import bsa
    c = s["c"]
    if c["norm"]:
        _, (codes, top) = bsa.gate_norm(s["x"][None], scale=s["scale"], shift=s["shift"], pre="rms", eps=1e-6, quantize=True)
    else:
        codes, top = bsa.quantize_int8(s["x"])
    return bsa.linear_int8(codes, top, s["w8"], s["w_scale"], bias=s["bias"], out_dtype=_TYPES[c["out"]])


def run(state):
    op = state["c"]["op"]
    if own:
        return {"rotary": _own_rotary, "norm": _own_norm, "linear": _own_linear}[op](state)
    return {"rotary": _plain_rotary, "norm": _plain_norm, "linear": _plain_linear}[op](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tensors"] * c["B"] * c["H"] * c["N"] * HEAD
        size = 4 if c["dtype"] == "fp32" else 2
        turned = min(2, c["tensors"]) * c["B"] * c["H"] * c["N"]
        return {"bytes": 2 * n * size + 4 * c["N"] * c["axes"] + 4 * c["r"],
                "flops": turned * (3 * c["r"] + (4 * HEAD if c["norm"] else 0))}
    if c["op"] == "norm":
        n, size = c["B"] * c["N"] * c["C"], 4 if c["stream"] == "fp32" else 2
        vec = {"none": 0, "batch": c["B"] * c["C"], "token": n}[c["mod"]]
        vec *= (3 if c["branch"] else 2) * (4 if c["mod_dtype"] == "fp32" else 2)
        own_bytes = (2 * size + 2 + 2) if c["branch"] else (size + 2)
        return {"bytes": n * own_bytes + vec, "flops": n * (14 if c["branch"] else 8)}
    M, K, N = c["M"], c["K"], c["N"]
    return {"bytes": 2 * M * K + N * K + 4 * N + M * N * (4 if c["out"] == "fp32" else 2), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64 bits

def _exact_rotary(c, seed):
    s = prepare(c, seed)
    ids = [a for a, n in enumerate(s["pairs"]) for _ in range(n)]
    out = [torch.empty(x.shape, dtype=torch.float64, device="cuda") for x in s["parts"]]
    for t0 in range(0, c["N"], 4_096):       # a slice of the tokens at a time
        t1 = min(c["N"], t0 + 4_096)
        angle = torch.stack([s["positions"][t0:t1, a].double() for a in ids], 1) * s["freqs"][None]
        turn = torch.polar(torch.full_like(angle, s["m"]), -angle if c["inverse"] else angle)
        for i, x in enumerate(s["parts"]):
            x = x[:, :, t0:t1].double().contiguous()
            if i < 2:
                if c["norm"]:
                    x = x / ((x * x).sum(-1, keepdim=True) / HEAD + 1e-6).sqrt() * s["weights"][i].double()
                r = c["r"]
                pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :r].unflatten(-1, (r // 2, 2))
                z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                x[..., :r] = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
            out[i][:, :, t0:t1] = x
    return out


def _exact_normed(v, kind, weight, bias):
    if kind == "layer":
        mean = v.sum(-1, keepdim=True) / v.shape[-1]
        v = (v - mean) / (((v - mean) ** 2).sum(-1, keepdim=True) / v.shape[-1] + 1e-6).sqrt()
    elif kind == "rms":
        v = v / ((v * v).sum(-1, keepdim=True) / v.shape[-1] + 1e-6).sqrt()
    v = v if weight is None else v * weight.double()
    return v if bias is None else v + bias.double()


def _exact_norm(c, seed):
    s = prepare(c, seed)
    h, z = (torch.empty(s["x"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    part = lambda v, t0, t1: v.double() if v.shape[1] == 1 else v[:, t0:t1].double()  # noqa: E731
    for t0 in range(0, c["N"], 8_192):
        t1 = min(c["N"], t0 + 8_192)
        v = s["x"][:, t0:t1].double()
        if s["y"] is not None:
            y = _exact_normed(s["y"][:, t0:t1].double(), c["post"], s["post_weight"], s["post_bias"])
            v = v + (y if s["gate"] is None else part(s["gate"], t0, t1) * y)
        h[:, t0:t1] = v
        u = _exact_normed(v, c["pre"], s["pre_weight"], s["pre_bias"])
        if s["scale"] is not None:
            u = u + u * part(s["scale"], t0, t1) + part(s["shift"], t0, t1)
        z[:, t0:t1] = u
    return {"h": h if s["y"] is not None else None, "z": z}


def _exact_linear(c, seed):
    s = prepare(c, seed)
    M, K, N = c["M"], c["K"], c["N"]
    x = s["x"][0].permute(1, 0, 2).reshape(M, K).double() if c["heads"] else s["x"].double()
    if c["norm"]:
        x = _exact_normed(x, "rms", None, None)
        x = x + x * s["scale"][0].double() + s["shift"][0].double()
    top = x.abs().max(1, keepdim=True).values.clamp(min=FLOOR)
    # the format: a 32-bit factor 127 / top, the 32-bit product rounded to the nearest whole number
    codes = (x * (127.0 / top).float().double()).float().round()
    total = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    w = s["w8"].float()
    for k in range(0, K, 1_024):             # 1,024 products of at most 127 x 127 stay below 2^24: each part is exact
        total += codes[:, k:k + 1_024] @ w[:, k:k + 1_024].t()
    total *= (top / 127.0).float().double() * s["w_scale"].double()
    if s["bias"] is not None:
        total += s["bias"].double()
    return total


def exact(case, seed):
    if case["op"] == "rotary":
        return _exact_rotary(case, seed)
    return _exact_norm(case, seed) if case["op"] == "norm" else _exact_linear(case, seed)
