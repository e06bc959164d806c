"""fp64 CPU oracle of the operators around the attention (test infrastructure only).

rotary positions with the per-head RMS norm, the gated and modulated norms, the int8 rows and the int8
product.  Plain numpy, one formula a function; the int8 format's fp32 factors are reproduced bit for bit.
"""

from __future__ import annotations

import math

import numpy as np

INT8_FLOOR = 2.0 ** -100


def rotary_freqs(pairs, base=10000.0, scaling="plain", factor=1.0, trained_length=0.0, fast_turns=32.0,
                 slow_turns=1.0):
    """(radians a position of every pair, factor on cos and sin)."""
    i = np.arange(pairs, dtype=np.float64)
    if scaling == "ntk" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1))
    f = np.exp(-math.log(base) * i / max(pairs, 1))
    if scaling == "linear":
        f = f / factor
    if scaling in ("yarn", "by_parts"):
        turns = trained_length * f / (2 * math.pi)
        keep = np.clip((turns - slow_turns) / (fast_turns - slow_turns), 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rms(v, eps):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def layer(v, eps):
    d = v - v.mean(-1, keepdims=True)
    return d / np.sqrt((d * d).mean(-1, keepdims=True) + eps)


def turns(positions, freqs):
    """Angles modulo 2 pi of whole positions [N, pairs], from exact integer products."""
    out = np.empty((len(positions), len(freqs)))
    for i, f in enumerate(freqs):
        num, den = float(f).as_integer_ratio()
        for n, p in enumerate(positions[:, i]):
            # p f as an exact fraction, reduced by whole turns with 200 bits of 2 pi
            q = (int(p) * num << 200) // den
            out[n, i] = float(q % TWO_PI_200) / 2.0 ** 200
    return out


# floor(2 pi 2^200): pi from Machin's formula 16 atan(1/5) - 4 atan(1/239) in whole numbers
def _atan_inv(n, one):
    total, term, k = 0, one // n, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


_ONE = 1 << 240
TWO_PI_200 = (2 * (16 * _atan_inv(5, _ONE) - 4 * _atan_inv(239, _ONE))) >> 40


def rotary(x, positions, freqs, layout, axis_pairs, weight=None, eps=1e-6, scale=1.0, inverse=False):
    """x [H, N, 128], positions [N, axes] -> the turned rows, fp64."""
    x = x.astype(np.float64)
    if weight is not None:
        x = rms(x, eps) * weight
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    theta = turns(positions[:, axis], freqs)
    if inverse:
        theta = -theta
    r = 2 * len(freqs)
    lo = np.arange(r // 2) if layout == "half" else 2 * np.arange(r // 2)
    hi = lo + (r // 2 if layout == "half" else 1)
    y = x.copy()
    y[..., lo] = scale * (x[..., lo] * np.cos(theta) - x[..., hi] * np.sin(theta))
    y[..., hi] = scale * (x[..., hi] * np.cos(theta) + x[..., lo] * np.sin(theta))
    return y


def gate_norm(x, y=None, gate=None, scale=None, shift=None, pre="rms", pre_weight=None, pre_bias=None,
              post="none", post_weight=None, post_bias=None, eps=1e-6, residual_scale=1.0,
              branch_scale=1.0):
    """(h, z) for rows [..., C]; gate, scale and shift broadcast."""
    def norm(v, kind, weight, bias):
        v = layer(v, eps) if kind == "layer" else (rms(v, eps) if kind == "rms" else v)
        v = v if weight is None else v * weight
        return v if bias is None else v + bias
    h = x.astype(np.float64)
    if y is not None:
        b = norm(y.astype(np.float64), post, post_weight, post_bias)
        h = residual_scale * h + branch_scale * (b if gate is None else gate * b)
    z = norm(h, pre, pre_weight, pre_bias)
    z = z if scale is None else z * (1.0 + scale)
    return h, (z if shift is None else z + shift)


def quantize_int8(x):
    """(codes, scales) of fp32-valued rows [M, K], every rounding as the format says."""
    x = x.astype(np.float32)
    amax = np.maximum(np.abs(x).max(1), np.float32(INT8_FLOOR))
    finite = np.isfinite(x).all(1)
    amax = np.where(finite, amax, np.float32(1.0)).astype(np.float32)
    inv = np.float32(127.0) / amax
    codes = np.rint(np.where(finite[:, None], x, np.float32(0)) * inv[:, None]).astype(np.int8)
    scales = np.where(finite, amax / np.float32(127.0), np.float32(np.nan)).astype(np.float32)
    return codes, scales


def linear_int8(a, a_scale, w, w_scale, bias=None):
    """fp64 product of int8 codes with their scales; the sum in whole numbers."""
    total = a.astype(np.int64) @ w.astype(np.int64).T
    out = total * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
    return out if bias is None else out + bias.astype(np.float64)
