"""Thin ctypes binding over libbsa.so (include/bsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch tensors (device memory + streams); the functions
keep the C names.  There is no fallback: if libbsa.so is missing or the
device is not sm_100 the call raises.
"""

from __future__ import annotations

import ctypes
import math
import operator
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsa.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "bsa.h")

(BSA_OK, BSA_ERR_INVALID, BSA_ERR_ALIGN, BSA_ERR_CUDA, BSA_ERR_TIMEOUT, BSA_ERR_UNSUPPORTED,
 BSA_ERR_SCRATCH) = range(7)
BSA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
VARIANTS = {"anchor": 0, "mean": 1}


class BsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class bsa_params(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
        ("D", ctypes.c_int32), ("top_k", ctypes.c_int32), ("prefix", ctypes.c_int32),
        ("variant", ctypes.c_int32), ("dev_status", ctypes.c_void_p),
    ]


class bsa_fp8_operands(ctypes.Structure):
    """Mirror of bsa_fp8_operands (include/bsa.h): e4m3 codes and fp32 scales."""
    _fields_ = [("q8", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("k8", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("vt8", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("ks8", ctypes.c_void_p), ("ks_scale", ctypes.c_void_p),
                ("vst8", ctypes.c_void_p), ("vs_scale", ctypes.c_void_p),
                ("v_ref", ctypes.c_void_p)]


DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.int8: 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "by_parts": 4}
NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class bsa_rotary_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "N", "D", "rotary_dim", "layout", "axes")]
                + [("axis_pairs", _i32 * 4)]
                + [(n, _i32) for n in ("inverse", "in_dtype", "out_dtype")]
                + [("scale", _f32), ("eps", _f32)]
                + [(n, _i64) for n in ("in_b", "in_h", "in_n", "out_b", "out_h", "out_n", "pos_b",
                                       "pos_n")])


class bsa_gate_norm_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "N", "C", "pre", "post", "x_dtype", "y_dtype",
                                     "mod_dtype", "z_dtype")]
                + [(n, _f32) for n in ("eps", "residual_scale", "branch_scale")]
                + [(n, _i64) for n in ("x_b", "x_n", "y_b", "y_n", "h_b", "h_n", "z_b", "z_n",
                                       "gate_b", "gate_n", "scale_b", "scale_n", "shift_b",
                                       "shift_n")] + [("dev_status", ctypes.c_void_p)])


class bsa_gate_norm_inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "y", "gate", "scale", "shift", "post_weight",
                                               "post_bias", "pre_weight", "pre_bias")]


class bsa_quantize_int8_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "N", "S", "L", "x_dtype")]
                + [(n, _i64) for n in ("x_b", "x_n", "x_s", "ld")])


class bsa_linear_int8_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("M", "N", "K", "out_dtype")]
                + [(n, _i64) for n in ("lda", "ldw", "ldo")] + [("dev_status", ctypes.c_void_p)])


class bsa_block_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("C", "x_dtype", "mod_dtype", "pre", "post")]
                + [(n, _f32) for n in ("eps", "residual_scale", "branch_scale", "qk_eps",
                                       "rope_scale")]
                + [(n, _i32) for n in ("rotary_dim", "layout", "axes")]
                + [("axis_pairs", _i32 * 4)]
                + [(n, _i64) for n in ("gate_b", "gate_n", "scale_b", "scale_n", "shift_b",
                                       "shift_n", "pos_b", "pos_n", "ld_qkv", "ld_out")])


class bsa_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "gate", "scale", "shift", "pre_weight", "pre_bias", "post_weight", "post_bias", "w_qkv",
        "s_qkv", "b_qkv", "w_out", "s_out", "b_out", "q_weight", "k_weight", "positions", "freqs")]


_lib = None
_P = ctypes.POINTER(bsa_params)
_F8 = ctypes.POINTER(bsa_fp8_operands)
_vp = ctypes.c_void_p
_SIGS = {
    "bsa_num_blocks": (ctypes.c_int32, [_P]),
    "bsa_select_capacity": (ctypes.c_int32, [_P]),
    "bsa_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_pool": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp]),
    "bsa_summarize": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_select": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp]),
    "bsa_attend": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_forward": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "bsa_forward_host": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, ctypes.c_size_t, _vp]),
    "bsa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bsa_debug_expired_wait": (ctypes.c_int, [_vp, ctypes.c_uint64, _vp]),
    "bsa_forward_noalloc": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_reblock_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_reblock": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "bsa_permute": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_pool_permuted": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_summarize_permuted": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _vp]),
    "bsa_unpermute": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_forward_reblock_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_forward_reblock": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                           _vp]),
    "bsa_fp8_operands_bytes": (ctypes.c_size_t, [_P]),
    "bsa_fp8_operands_carve": (ctypes.c_int, [_P, _vp, ctypes.c_size_t, _F8]),
    "bsa_quantize_fp8": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _F8, _vp]),
    "bsa_attend_fp8": (ctypes.c_int, [_P, _F8, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bsa_forward_fp8_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_forward_fp8": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "bsa_threshold_capacity": (ctypes.c_int32, [_P]),
    "bsa_select_threshold": (ctypes.c_int, [_P, ctypes.c_float, _vp, _vp, _vp, _vp, _vp]),
    "bsa_attend_lists_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_attend_lists": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, ctypes.c_int32, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "bsa_forward_threshold_workspace_bytes": (ctypes.c_size_t, [_P]),
    "bsa_forward_threshold": (ctypes.c_int, [_P, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp,
                                             ctypes.c_size_t, _vp]),
    "bsa_extra_side_capacity": (ctypes.c_int32, [_P, ctypes.c_int32]),
    "bsa_summarize_stats": (ctypes.c_int, [_P] + [_vp] * 11),
    "bsa_select_extra_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int32]),
    "bsa_select_extra": (ctypes.c_int, [_P, ctypes.c_int32] + [_vp] * 7 + [ctypes.c_size_t, _vp]),
    "bsa_extra_summaries": (ctypes.c_int, [_P, ctypes.c_int32] + [_vp] * 15),
    "bsa_attend_extra": (ctypes.c_int, [_P, ctypes.c_int32] + [_vp] * 17),
    "bsa_forward_extra_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int32]),
    "bsa_forward_extra": (ctypes.c_int, [_P, ctypes.c_int32] + [_vp] * 6 + [ctypes.c_size_t, _vp]),
}
_HOST12 = [_vp] * 11 + [ctypes.c_size_t, _vp]
_SIGS["bsa_forward_fp8_host"] = (ctypes.c_int, [_P] + _HOST12)
_SIGS["bsa_forward_threshold_host"] = (ctypes.c_int, [_P, ctypes.c_float] + _HOST12)
_SIGS["bsa_forward_extra_host"] = (ctypes.c_int, [_P, ctypes.c_int32] + _HOST12)
_SIGS["bsa_forward_reblock_host"] = (ctypes.c_int, [_P] + _HOST12)
_SIGS["bsa_rotary_freqs"] = (ctypes.c_int, [_i32, ctypes.c_double, _i32] + [ctypes.c_double] * 4
                             + [_vp, _vp])
_SIGS["bsa_rotary"] = (ctypes.c_int, [ctypes.POINTER(bsa_rotary_params)] + [_vp] * 11)
_SIGS["bsa_rotary_each"] = _SIGS["bsa_rotary"]
_SIGS["bsa_gate_norm"] = (ctypes.c_int, [ctypes.POINTER(bsa_gate_norm_params),
                                         ctypes.POINTER(bsa_gate_norm_inputs)] + [_vp] * 4)
_SIGS["bsa_quantize_int8"] = (ctypes.c_int, [ctypes.POINTER(bsa_quantize_int8_params)] + [_vp] * 4)
_SIGS["bsa_linear_int8"] = (ctypes.c_int, [ctypes.POINTER(bsa_linear_int8_params)] + [_vp] * 7)
_BP = ctypes.POINTER(bsa_block_params)
_SIGS["bsa_forward_block_workspace_bytes"] = (ctypes.c_size_t, [_P, _BP])
_SIGS["bsa_forward_block"] = (ctypes.c_int, [_P, _BP, ctypes.POINTER(bsa_block_weights)]
                              + [_vp] * 3 + [ctypes.c_size_t, _vp])
BSA_MAX_EXTRA_TOKENS = 512


def lib() -> ctypes.CDLL:
    """Load libbsa.so once (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m "
                               "block_sparse_video_bsa_b200.build` first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        L.addresses = {name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value
                       for name in _SIGS}
        _lib = L
    return _lib


def header_functions() -> list:
    """Names of the functions include/bsa.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bsa_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().bsa_status_string(int(status)).decode()


def params(B, H, N, top_k, prefix=0, variant="anchor", D=128, dev_status=None) -> bsa_params:
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    ds = None if dev_status is None else dev_status.data_ptr()
    return bsa_params(B, H, N, D, top_k, prefix, v, ds)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc, where):
    if rc != BSA_OK:
        raise BsaError(rc, where)


# --------------------------------------------------------------- sizes

def bsa_num_blocks(p: bsa_params) -> int:
    return lib().bsa_num_blocks(ctypes.byref(p))


def bsa_select_capacity(p: bsa_params) -> int:
    return lib().bsa_select_capacity(ctypes.byref(p))


def bsa_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_workspace_bytes(ctypes.byref(p))


# --------------------------------------------------------------- stages

def bsa_pool(p, Q, qpool, anchor, stream=None):
    _check(lib().bsa_pool(ctypes.byref(p), _ptr(Q), _ptr(qpool), _ptr(anchor), _stream(stream)),
           "bsa_pool")


def bsa_summarize(p, K, V, anchor, kpool, ksum, vsum, bias, stream=None):
    _check(lib().bsa_summarize(ctypes.byref(p), _ptr(K), _ptr(V), _ptr(anchor), _ptr(kpool),
                               _ptr(ksum), _ptr(vsum), _ptr(bias), _stream(stream)),
           "bsa_summarize")


def bsa_select(p, qpool, kpool, idx, cnt, stream=None):
    _check(lib().bsa_select(ctypes.byref(p), _ptr(qpool), _ptr(kpool), _ptr(idx), _ptr(cnt),
                            _stream(stream)), "bsa_select")


def bsa_attend(p, Q, K, V, idx, cnt, ksum, vsum, bias, O, lse=None, stream=None):
    _check(lib().bsa_attend(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(cnt),
                            _ptr(ksum), _ptr(vsum), _ptr(bias), _ptr(O), _ptr(lse),
                            _stream(stream)), "bsa_attend")


def bsa_forward(p, Q, K, V, O, lse, workspace, stream=None):
    _check(lib().bsa_forward(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream)), "bsa_forward")


def bsa_forward_host(p, hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream=None):
    _check(lib().bsa_forward_host(ctypes.byref(p), _ptr(hQ), _ptr(hK), _ptr(hV), _ptr(hO),
                                  _ptr(hlse), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dO), _ptr(dlse),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "bsa_forward_host")


def _host_args(hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream):
    return (_ptr(hQ), _ptr(hK), _ptr(hV), _ptr(hO), _ptr(hlse), _ptr(dQ), _ptr(dK), _ptr(dV),
            _ptr(dO), _ptr(dlse), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream))


def bsa_forward_fp8_host(p, hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream=None):
    _check(lib().bsa_forward_fp8_host(ctypes.byref(p), *_host_args(
        hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream)), "bsa_forward_fp8_host")


def bsa_forward_threshold_host(p, tau, hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace,
                               stream=None):
    _check(lib().bsa_forward_threshold_host(ctypes.byref(p), float(tau), *_host_args(
        hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream)),
        "bsa_forward_threshold_host")


def bsa_forward_extra_host(p, n_extra, hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace,
                           stream=None):
    _check(lib().bsa_forward_extra_host(ctypes.byref(p), int(n_extra), *_host_args(
        hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream)), "bsa_forward_extra_host")


def bsa_forward_reblock_host(p, hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace,
                             stream=None):
    _check(lib().bsa_forward_reblock_host(ctypes.byref(p), *_host_args(
        hQ, hK, hV, hO, hlse, dQ, dK, dV, dO, dlse, workspace, stream)),
        "bsa_forward_reblock_host")


def bsa_forward_noalloc(p, Q, K, V, O, lse=None, stream=None):
    """bsa_forward with its workspace in the library's static device scratch,
    for callers that cannot allocate device memory (see include/bsa.h)."""
    _check(lib().bsa_forward_noalloc(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                     _ptr(lse), _stream(stream)), "bsa_forward_noalloc")


def bsa_reblock_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_reblock_workspace_bytes(ctypes.byref(p))


def bsa_reblock(p, Q, K, perm, workspace, stream=None):
    _check(lib().bsa_reblock(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(perm), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)),
           "bsa_reblock")


def bsa_pool_permuted(p, Q, perm, Qp, qpool, anchor, stream=None):
    _check(lib().bsa_pool_permuted(ctypes.byref(p), _ptr(Q), _ptr(perm), _ptr(Qp), _ptr(qpool),
                                   _ptr(anchor), _stream(stream)), "bsa_pool_permuted")


def bsa_summarize_permuted(p, K, V, perm, Kp, Vp, anchor, kpool, ksum, vsum, bias, stream=None):
    _check(lib().bsa_summarize_permuted(ctypes.byref(p), _ptr(K), _ptr(V), _ptr(perm), _ptr(Kp),
                                        _ptr(Vp), _ptr(anchor), _ptr(kpool), _ptr(ksum),
                                        _ptr(vsum), _ptr(bias), _stream(stream)),
           "bsa_summarize_permuted")


def bsa_permute(p, Q, K, V, perm, Qp, Kp, Vp, stream=None):
    _check(lib().bsa_permute(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(perm), _ptr(Qp),
                             _ptr(Kp), _ptr(Vp), _stream(stream)), "bsa_permute")


def bsa_unpermute(p, Op, lsep, perm, O, lse=None, stream=None):
    _check(lib().bsa_unpermute(ctypes.byref(p), _ptr(Op), _ptr(lsep), _ptr(perm), _ptr(O),
                               _ptr(lse), _stream(stream)), "bsa_unpermute")


def bsa_forward_reblock_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_forward_reblock_workspace_bytes(ctypes.byref(p))


def bsa_forward_reblock(p, Q, K, V, O, lse, workspace, stream=None):
    _check(lib().bsa_forward_reblock(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                     _ptr(lse), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "bsa_forward_reblock")


def reblock(Q, K, prefix=0, stream=None):
    """perm [B, H, N] int32 of the reblocked layout (see bsa_reblock)."""
    B, H, N, D = Q.shape
    p = params(B, H, N, 1, prefix, D=D)
    perm = torch.empty(B, H, N, dtype=torch.int32, device=Q.device)
    ws = torch.empty(max(256, bsa_reblock_workspace_bytes(p)), dtype=torch.uint8, device=Q.device)
    bsa_reblock(p, Q, K, perm, ws, stream)
    return perm


def forward_reblock(Q, K, V, top_k, prefix=0, variant="anchor", return_lse=False, ws=None,
                    stream=None):
    """bsa_forward_reblock: block-sparse attention on the reblocked layout,
    O (and lse) returned in the original token order."""
    B, H, N, D = Q.shape
    p = params(B, H, N, top_k, prefix, variant, D=D)
    O = torch.empty_like(Q)
    lse = torch.empty(B, H, N, dtype=torch.float32, device=Q.device) if return_lse else None
    if ws is None:
        ws = torch.empty(bsa_forward_reblock_workspace_bytes(p), dtype=torch.uint8,
                         device=Q.device)
    bsa_forward_reblock(p, Q, K, V, O, lse, ws, stream)
    return (O, lse) if return_lse else O


def bsa_fp8_operands_bytes(p: bsa_params) -> int:
    return lib().bsa_fp8_operands_bytes(ctypes.byref(p))


def bsa_fp8_operands_carve(p, buf) -> bsa_fp8_operands:
    ops = bsa_fp8_operands()
    _check(lib().bsa_fp8_operands_carve(ctypes.byref(p), _ptr(buf), buf.numel() * buf.element_size(),
                                        ctypes.byref(ops)), "bsa_fp8_operands_carve")
    return ops


def bsa_quantize_fp8(p, Q, K, V, ksum, vsum, ops, stream=None):
    _check(lib().bsa_quantize_fp8(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(ksum),
                                  _ptr(vsum), ctypes.byref(ops), _stream(stream)),
           "bsa_quantize_fp8")


def bsa_attend_fp8(p, ops, idx, cnt, bias, O, lse=None, stream=None):
    _check(lib().bsa_attend_fp8(ctypes.byref(p), ctypes.byref(ops), _ptr(idx), _ptr(cnt),
                                _ptr(bias), _ptr(O), _ptr(lse), _stream(stream)), "bsa_attend_fp8")


def bsa_forward_fp8_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_forward_fp8_workspace_bytes(ctypes.byref(p))


def bsa_forward_fp8(p, Q, K, V, O, lse, workspace, stream=None):
    _check(lib().bsa_forward_fp8(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "bsa_forward_fp8")


def bsa_threshold_capacity(p: bsa_params) -> int:
    return lib().bsa_threshold_capacity(ctypes.byref(p))


def bsa_select_threshold(p, tau, qpool, kpool, idx, cnt, stream=None):
    _check(lib().bsa_select_threshold(ctypes.byref(p), float(tau), _ptr(qpool), _ptr(kpool),
                                      _ptr(idx), _ptr(cnt), _stream(stream)),
           "bsa_select_threshold")


def bsa_attend_lists_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_attend_lists_workspace_bytes(ctypes.byref(p))


def bsa_attend_lists(p, Q, K, V, idx, cnt, ksum, vsum, bias, O, lse, workspace, stream=None):
    """bsa_attend over variable-length lists; the row stride is idx's last dimension."""
    _check(lib().bsa_attend_lists(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx),
                                  int(idx.shape[-1]), _ptr(cnt), _ptr(ksum), _ptr(vsum),
                                  _ptr(bias), _ptr(O), _ptr(lse), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
           "bsa_attend_lists")


def bsa_forward_threshold_workspace_bytes(p: bsa_params) -> int:
    return lib().bsa_forward_threshold_workspace_bytes(ctypes.byref(p))


def bsa_forward_threshold(p, tau, Q, K, V, O, lse, workspace, stream=None):
    _check(lib().bsa_forward_threshold(ctypes.byref(p), float(tau), _ptr(Q), _ptr(K), _ptr(V),
                                       _ptr(O), _ptr(lse), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream)), "bsa_forward_threshold")


def bsa_extra_side_capacity(p: bsa_params, n_extra: int) -> int:
    return lib().bsa_extra_side_capacity(ctypes.byref(p), int(n_extra))


def bsa_summarize_stats(p, K, V, anchor, kpool, ksum, vsum, bias, kstat, vstat, lse_blk,
                        stream=None):
    _check(lib().bsa_summarize_stats(ctypes.byref(p), _ptr(K), _ptr(V), _ptr(anchor), _ptr(kpool),
                                     _ptr(ksum), _ptr(vsum), _ptr(bias), _ptr(kstat), _ptr(vstat),
                                     _ptr(lse_blk), _stream(stream)), "bsa_summarize_stats")


def bsa_select_extra_workspace_bytes(p: bsa_params, n_extra: int) -> int:
    return lib().bsa_select_extra_workspace_bytes(ctypes.byref(p), int(n_extra))


def bsa_select_extra(p, n_extra, qpool, K, idx, cnt, extra, ecnt, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().bsa_select_extra(ctypes.byref(p), int(n_extra), _ptr(qpool), _ptr(K), _ptr(idx),
                                  _ptr(cnt), _ptr(extra), _ptr(ecnt), _ptr(workspace), nbytes,
                                  _stream(stream)), "bsa_select_extra")


def bsa_extra_summaries(p, n_extra, K, V, anchor, kpool, kstat, vstat, lse_blk, extra, ecnt,
                        side_k, side_v, side_bias, side_blk, side_cnt, stream=None):
    _check(lib().bsa_extra_summaries(ctypes.byref(p), int(n_extra), _ptr(K), _ptr(V), _ptr(anchor),
                                     _ptr(kpool), _ptr(kstat), _ptr(vstat), _ptr(lse_blk),
                                     _ptr(extra), _ptr(ecnt), _ptr(side_k), _ptr(side_v),
                                     _ptr(side_bias), _ptr(side_blk), _ptr(side_cnt),
                                     _stream(stream)), "bsa_extra_summaries")


def bsa_attend_extra(p, n_extra, Q, K, V, idx, cnt, extra, ecnt, ksum, vsum, bias, side_k, side_v,
                     side_bias, side_cnt, O, lse=None, stream=None):
    _check(lib().bsa_attend_extra(ctypes.byref(p), int(n_extra), _ptr(Q), _ptr(K), _ptr(V),
                                  _ptr(idx), _ptr(cnt), _ptr(extra), _ptr(ecnt), _ptr(ksum),
                                  _ptr(vsum), _ptr(bias), _ptr(side_k), _ptr(side_v),
                                  _ptr(side_bias), _ptr(side_cnt), _ptr(O), _ptr(lse),
                                  _stream(stream)), "bsa_attend_extra")


def bsa_forward_extra_workspace_bytes(p: bsa_params, n_extra: int) -> int:
    return lib().bsa_forward_extra_workspace_bytes(ctypes.byref(p), int(n_extra))


def bsa_forward_extra(p, n_extra, Q, K, V, O, lse, workspace, stream=None):
    _check(lib().bsa_forward_extra(ctypes.byref(p), int(n_extra), _ptr(Q), _ptr(K), _ptr(V),
                                   _ptr(O), _ptr(lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "bsa_forward_extra")


def extra_buffers(B, H, N, top_k, n_extra, prefix=0, variant="anchor", device="cuda"):
    """Device tensors for the extra-token stages (statistics, lists, side
    table, candidate scratch)."""
    p = params(B, H, N, top_k, prefix, variant)
    nb = bsa_num_blocks(p)
    scap = bsa_extra_side_capacity(p, n_extra)
    if nb < 0 or scap < 0:
        raise BsaError(BSA_ERR_INVALID, "extra_buffers")
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    return dict(
        kstat=torch.empty(B, H, nb, 128, dtype=f32, device=device),
        vstat=torch.empty(B, H, nb, 128, dtype=f32, device=device),
        lse_blk=torch.empty(B, H, nb, dtype=f32, device=device),
        extra=torch.empty(B, H, nb, max(n_extra, 1), dtype=i32, device=device),
        ecnt=torch.empty(B, H, nb, dtype=i32, device=device),
        side_k=torch.empty(B, H, nb, max(scap, 1), 128, dtype=bf16, device=device),
        side_v=torch.empty(B, H, nb, max(scap, 1), 128, dtype=bf16, device=device),
        side_bias=torch.empty(B, H, nb, max(scap, 1), dtype=f32, device=device),
        side_blk=torch.empty(B, H, nb, max(scap, 1), dtype=i32, device=device),
        side_cnt=torch.empty(B, H, nb, dtype=i32, device=device),
        cand=torch.empty(max(256, bsa_select_extra_workspace_bytes(p, n_extra)), dtype=torch.uint8,
                         device=device),
    )


def forward_extra(Q, K, V, top_k, n_extra, prefix=0, variant="anchor", return_lse=False, ws=None,
                  stream=None):
    """bsa_forward_extra: block-sparse attention plus n_extra top-scoring
    tokens per query block."""
    B, H, N, D = Q.shape
    p = params(B, H, N, top_k, prefix, variant, D=D)
    O = torch.empty_like(Q)
    lse = torch.empty(B, H, N, dtype=torch.float32, device=Q.device) if return_lse else None
    if ws is None:
        ws = torch.empty(bsa_forward_extra_workspace_bytes(p, n_extra), dtype=torch.uint8,
                         device=Q.device)
    bsa_forward_extra(p, n_extra, Q, K, V, O, lse, ws, stream)
    return (O, lse) if return_lse else O


def bsa_debug_expired_wait(dev_status, timeout_ns: int, stream=None):
    _check(lib().bsa_debug_expired_wait(_ptr(dev_status), int(timeout_ns), _stream(stream)),
           "bsa_debug_expired_wait")


# --------------------------------------------------------------- around the attention
#
# A call on one token is a few microseconds on the GPU, so these wrappers keep
# the host's share small: checks of shapes, strides and types and the filled
# parameter struct are a pure function of the arguments' layout and are kept
# per layout (never per address); a repeated layout costs a lookup, the output
# allocations and the launch, which csrc/host.cpp does (norm of one row: 13.5 us
# a call in Python alone, 8.4 with it).

_host = None


def _load_host():
    """The extension module built from csrc/host.cpp (raises if it was not built, or for another
    torch or Python)."""
    global _host
    if _host is None:
        from .build import host_built_for
        again = "run `python -m block_sparse_video_bsa_b200.build`"
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_host.so")):
            raise RuntimeError(f"_host.so is missing: {again} first")
        try:
            from . import _host as module
        except ImportError as e:      # a symbol of another torch
            raise RuntimeError(f"_host.so does not load ({e}): {again} again") from e
        if getattr(module, "built_for", None) != host_built_for():
            raise RuntimeError(f"_host.so was built for {getattr(module, 'built_for', 'another torch')}, this is "
                               f"{host_built_for()}: {again} again")
        _host = module
    return _host


def _keep(plans, key, plan):
    """Remember a layout's plan; a program has a handful of them."""
    if len(plans) >= 256:
        plans.clear()
    plans[key] = plan
    return plan


_rotary_plans, _gate_norm_plans, _quantize_plans, _linear_plans = {}, {}, {}, {}


def _need(ok, where):
    if not ok:
        raise BsaError(BSA_ERR_INVALID, where)


def _sig(t):
    """What a plan may depend on: a tensor's layout, never its address."""
    return None if t is None else (t.dtype, t.shape, t.stride(), t.get_device())


def _one_device(where, ref, *sigs):
    """The CUDA device of every given tensor."""
    _need(ref[3] >= 0, where)
    for g in sigs:
        _need(g is None or g[3] == ref[3], where)
    return ref[3]


def _elsewhere(device, stream, where):
    """Context in which `device` is current and outputs belong to `stream`."""
    if stream is None:
        return torch.cuda.device(device)
    _need(stream.device.index == device, where)
    return torch.cuda.stream(stream)


# torch's own accessors; the public ones where a torch lacks these (a few tenths of a us more)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _here(device, stream):
    return stream is None and _device_now() == device


def _vector(g, n, where):
    """An fp32 vector of n contiguous values, or None."""
    _need(g is None or (g[0] is torch.float32 and g[1] == (n,) and (n == 1 or g[2] == (1,))), where)


def _addr(t):
    return None if t is None else t.data_ptr()


_FLOATS = (torch.bfloat16, torch.float32)


def _packed(shape):
    """Strides of a contiguous tensor."""
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= max(d, 1)
    return tuple(reversed(strides))


def rotary_freqs(pairs, base=10000.0, scaling="plain", factor=1.0, trained_length=0,
                 fast_turns=32.0, slow_turns=1.0, device="cuda"):
    """(freqs, scale) for ``rotary``: radians a position of every pair (fp64 tensor) and the factor
    on cos and sin.  ``pairs`` is a number, or a list with one number an axis (the axes' frequencies
    one after another).  See bsa_rotary_freqs for the scalings."""
    scale = ctypes.c_float()
    out = []
    for n in ([pairs] if isinstance(pairs, int) else pairs):
        f = (ctypes.c_double * max(n, 1))()
        _check(lib().bsa_rotary_freqs(n, float(base), ROPE_SCALINGS[scaling], float(factor),
                                      float(trained_length), float(fast_turns), float(slow_turns),
                                      ctypes.byref(f), ctypes.byref(scale)), "bsa_rotary_freqs")
        out += list(f)[:n]
    return torch.tensor(out, dtype=torch.float64, device=device), scale.value


def _rotary_plan(parts, outs, pos, fr, weights, layout, pairs, eps, scale, inverse, out_dtype):
    """(device, output shapes and types, the filled structs of q, k and v, the address and the entry to
    call with it): one struct where the given tensors share their layout."""
    where = "rotary"
    given = [g for g in parts if g is not None]
    _need(given and len(outs) == 3 and pos is not None and fr is not None, where)
    device = _one_device(where, given[0], *given, *outs, pos, fr, *weights)
    B, N = given[0][1][0], given[0][1][2]
    for dtype, shape, stride, _ in given:
        _need(dtype in _FLOATS and len(shape) == 4 and shape[0] == B and shape[2] == N
              and shape[3] == 128 and stride[3] == 1, where)
    _need(fr[0] is torch.float64 and len(fr[1]) == 1 and (fr[1][0] <= 1 or fr[2] == (1,)), where)
    pairs = (fr[1][0],) if pairs is None else pairs
    _need(1 <= len(pairs) <= 4 and sum(pairs) == fr[1][0], where)
    pdtype, pshape, pstride, _ = pos
    if len(pshape) == 1:
        pshape, pstride = (*pshape, 1), (*pstride, 1)
    _need(pdtype is torch.int32 and len(pshape) in (2, 3) and pshape[-2:] == (N, len(pairs))
          and (pshape[-1] == 1 or pstride[-1] == 1)
          and (len(pshape) == 2 or pshape[0] in (1, B)), where)
    pos_b = pstride[0] if len(pshape) == 3 and pshape[0] > 1 else 0
    for g in weights:
        _vector(g, 128, where)
    want, kinds = [], {}
    for i, (x, y) in enumerate(zip(parts, outs)):
        if x is None:
            _need(y is None, where)
            want.append(None)
            continue
        dtype, shape, stride, _ = x
        H = shape[1]
        if y is None:
            y = (out_dtype or dtype, shape, (H * N * 128, N * 128, 128, 1), device)
        _need(y[0] in _FLOATS and y[1] == shape and y[2][3] == 1, where)
        want.append((tuple(y[1]), _packed(y[1]), y[0]))
        kinds.setdefault((H, stride, dtype, y[2], y[0]), []).append(i)
    each = (bsa_rotary_params * 3)()
    for (H, stride, dtype, ostride, odtype), ids in kinds.items():
        for i in ids:
            each[i] = bsa_rotary_params(B, H, N, 128, 2 * fr[1][0], ROPE_LAYOUTS[layout],
                                        len(pairs), (_i32 * 4)(*pairs), int(inverse), DTYPES[dtype],
                                        DTYPES[odtype], scale, eps, *stride[:3], *ostride[:3], pos_b,
                                        pstride[-2])
    if len(kinds) > 1:
        return device, tuple(want), each, ctypes.addressof(each), "bsa_rotary_each"
    return device, tuple(want), each, ctypes.addressof(each[i]), "bsa_rotary"


def rotary(q, k, v, positions, freqs, layout="half", axis_pairs=None, q_weight=None, k_weight=None,
           eps=1e-6, scale=1.0, inverse=False, out=None, out_dtype=None, stream=None):
    """bsa_rotary: (Q, K, V) as [B, H, N, 128] from q, k, v viewed as [B, H, N, 128] with any
    strides (token-major projections: ``qkv[:, :, 0].transpose(1, 2)`` and so on).

    Any of q, k, v may be None.  positions int32 [N, axes] or [B, N, axes] ([N] for one axis),
    freqs fp64 [pairs] from ``rotary_freqs``; axis_pairs lists the pairs of each axis.  k and v may
    have another head count than q.  ``out`` gives the outputs (a tensor may be its own output)."""
    outs = out if out is not None else (None, None, None)
    # plain numbers: a key that held the caller's object (a tensor of no dimension) would
    # match by identity and keep its first value
    if type(eps) is not float or type(scale) is not float or type(inverse) is not bool:
        eps, scale, inverse = float(eps), float(scale), bool(inverse)
    if axis_pairs is not None:
        axis_pairs = tuple(map(operator.index, axis_pairs))
    host = _host or _load_host()
    key = (host.layout(q, k, v, *outs, positions, freqs, q_weight, k_weight), layout, axis_pairs,
           eps, scale, inverse, out_dtype)
    plan = _rotary_plans.get(key)
    if plan is None:
        plan = _keep(_rotary_plans, key, _rotary_plan(
            (_sig(q), _sig(k), _sig(v)), tuple([_sig(y) for y in outs]), _sig(positions),
            _sig(freqs), (_sig(q_weight), _sig(k_weight)), layout, axis_pairs, eps, scale,
            inverse, out_dtype))
    device, want, _, p, name = plan
    if stream is not None or _device_now() != device:
        with _elsewhere(device, stream, "rotary"):
            return rotary(q, k, v, positions, freqs, layout, axis_pairs, q_weight, k_weight, eps,
                          scale, inverse, out, out_dtype)
    Q, K, V = [y if w is None or y is not None else host.empty(*w, freqs)
               for w, y in zip(want, outs)]
    rc = host.call(lib().addresses[name], p, q, k, v, positions, freqs,
                   q_weight if q is not None else None, k_weight if k is not None else None, Q, K, V,
                   _raw_stream(device))
    if rc:
        raise BsaError(rc, name)
    return Q, K, V


def _mod(g, B, N, C, where):
    """(batch stride, token stride) of a vector [C], [B or 1, C] or [B or 1, N or 1, C]."""
    if g is None:
        return 0, 0
    _, shape, stride, _ = g
    _need(1 <= len(shape) <= 3 and shape[-1] == C and (C == 1 or stride[-1] == 1), where)
    if len(shape) == 1:
        return 0, 0
    _need(shape[0] in (1, B) and (len(shape) == 2 or shape[1] in (1, N)), where)
    return (stride[0] if shape[0] > 1 else 0,
            stride[1] if len(shape) == 3 and shape[1] > 1 else 0)


def _rows(g, C):
    """Strides (batch, token) of rows [B, N, C]."""
    return (0, 0) if g is None else (g[2][0], g[2][1])


def _gate_norm_plan(x, y, gate, scale, shift, vectors, h_out, pre, post, eps, residual_scale,
                    branch_scale, quantize, z_dtype, want_z):
    where = "gate_norm"
    device = _one_device(where, x, y, gate, scale, shift, *vectors, h_out)
    _need(len(x[1]) == 3 and pre in NORMS and post in NORMS and z_dtype in _FLOATS, where)
    B, N, C = x[1]
    for g in (x, y, h_out):
        _need(g is None or (g[0] in _FLOATS and g[1] == x[1] and (C == 1 or g[2][2] == 1)), where)
    _need(h_out is None or (y is not None and h_out[0] is x[0]), where)
    mods = [g[0] for g in (gate, scale, shift) if g is not None]
    for dtype in mods:
        _need(dtype in _FLOATS and dtype is mods[0], where)
    for g in vectors:
        _vector(g, C, where)
    ld = -(-C // 16) * 16 if quantize else C
    h = (N * C, C) if h_out is None else _rows(h_out, C)
    p = bsa_gate_norm_params(
        B, N, C, NORMS[pre], NORMS[post], DTYPES[x[0]], DTYPES[y[0]] if y else 0,
        DTYPES[mods[0]] if mods else 1, 2 if quantize and want_z else DTYPES[z_dtype], eps,
        residual_scale, branch_scale, *_rows(x, C), *_rows(y, C), *h, N * ld, ld,
        *_mod(gate, B, N, C, where), *_mod(scale, B, N, C, where), *_mod(shift, B, N, C, where))
    return (device, p, ctypes.addressof(p), ((B, N, C), (N * C, C, 1)), ((B * N, C), (ld, 1)),
            ((B * N,), (1,)))


def gate_norm(x, y=None, gate=None, scale=None, shift=None, pre="rms", pre_weight=None,
              pre_bias=None, post="none", post_weight=None, post_bias=None, eps=1e-6,
              residual_scale=1.0, branch_scale=1.0, quantize=False, z_dtype=torch.bfloat16,
              h_out=None, want_z=True, dev_status=None, stream=None):
    """bsa_gate_norm: (h, z) with h = residual_scale x + branch_scale gate post(y) (x itself without
    y) and z = pre(h) (1 + scale) + shift.

    x, y [B, N, C]; gate, scale, shift [C], [B, C], [B, 1, C] or [B, N, C]; weights and biases fp32
    [C].  quantize: z is (codes [B N, C] int8, scales [B N]) for ``linear_int8``.  h_out: where h
    goes (x for an update in place).  want_z=False: z is None and only h is made."""
    host = _host or _load_host()
    if (type(eps) is not float or type(residual_scale) is not float
            or type(branch_scale) is not float or type(quantize) is not bool
            or type(want_z) is not bool):                # plain values in the key, as in rotary
        eps, residual_scale, branch_scale = float(eps), float(residual_scale), float(branch_scale)
        quantize, want_z = bool(quantize), bool(want_z)
    key = (host.layout(x, y, gate, scale, shift, post_weight, post_bias, pre_weight, pre_bias,
                       h_out), pre, post, eps, residual_scale, branch_scale, quantize, z_dtype,
           want_z)
    plan = _gate_norm_plans.get(key)
    if plan is None:
        plan = _keep(_gate_norm_plans, key, _gate_norm_plan(
            _sig(x), _sig(y), _sig(gate), _sig(scale), _sig(shift),
            (_sig(post_weight), _sig(post_bias), _sig(pre_weight), _sig(pre_bias)), _sig(h_out),
            pre, post, eps, residual_scale, branch_scale, quantize, z_dtype, want_z))
    device, p, ref, rows, codes, scales = plan
    if stream is not None or _device_now() != device:
        with _elsewhere(device, stream, "gate_norm"):
            return gate_norm(x, y, gate, scale, shift, pre, pre_weight, pre_bias, post, post_weight,
                             post_bias, eps, residual_scale, branch_scale, quantize, z_dtype, h_out,
                             want_z, dev_status)
    if dev_status is not None:
        _need(dev_status.get_device() == device, "gate_norm")
        p = bsa_gate_norm_params.from_buffer_copy(p)
        p.dev_status = dev_status.data_ptr()
        ref = ctypes.addressof(p)
    h, z, zs = h_out, None, None
    if h is None and y is not None:
        h = host.empty(*rows, x.dtype, x)
    if want_z and quantize:
        z, zs = host.empty(*codes, torch.int8, x), host.empty(*scales, torch.float32, x)
    elif want_z:
        z = host.empty(*rows, z_dtype, x)
    rc = host.call(lib().addresses["bsa_gate_norm"], ref,
                   (x, y, gate, scale, shift, post_weight, post_bias, pre_weight, pre_bias), h, z,
                   zs, _raw_stream(device))
    if rc:
        raise BsaError(rc, "bsa_gate_norm")
    return (x if h is None else h), (z if zs is None else (z, zs))


def _quantize_int8_plan(x):
    where = "quantize_int8"
    device = _one_device(where, x)
    dtype, shape, st, _ = x
    _need(dtype in _FLOATS and 2 <= len(shape) <= 4 and (shape[-1] == 1 or st[-1] == 1), where)
    if len(shape) == 4:
        (B, S, N, L), s = shape, (st[0], st[2], st[1])
    elif len(shape) == 3:
        (B, N, L), S, s = shape, 1, (st[0], st[1], 0)
    else:
        B, (N, L), S, s = 1, shape, 1, (0, st[0], 0)
    K = S * L
    ld = -(-K // 16) * 16
    p = bsa_quantize_int8_params(B, N, S, L, DTYPES[dtype], *s, ld)
    return device, p, ctypes.addressof(p), ((B * N, K), (ld, 1)), ((B * N,), (1,))


def quantize_int8(x, stream=None):
    """bsa_quantize_int8: (codes, scales) of the rows of x [M, K] or [B, N, K], or of the token rows
    of an attention output [B, H, N, D] (H D values a token).  codes int8 [rows, K] (row stride a
    multiple of 16), scales fp32 [rows]."""
    host = _host or _load_host()
    key = host.layout(x)
    plan = _quantize_plans.get(key)
    if plan is None:
        plan = _keep(_quantize_plans, key, _quantize_int8_plan(_sig(x)))
    device, _, p, rows, scales = plan
    if not _here(device, stream):
        with _elsewhere(device, stream, "quantize_int8"):
            return quantize_int8(x)
    codes, scale = host.empty(*rows, torch.int8, x), host.empty(*scales, torch.float32, x)
    _check(host.call(lib().addresses["bsa_quantize_int8"], p, x, codes, scale,
                     _raw_stream(device)), "bsa_quantize_int8")
    return codes, scale


def _linear_int8_plan(a, a_scale, w, w_scale, bias, out, out_dtype):
    where = "linear_int8"
    device = _one_device(where, a, a_scale, w, w_scale, bias, out)
    for g in (a, w):
        _need(g[0] is torch.int8 and len(g[1]) == 2 and (g[1][1] == 1 or g[2][1] == 1), where)
    _need(a[1][1] == w[1][1] and a_scale is not None and w_scale is not None, where)
    (M, K), N = a[1], w[1][0]
    _vector(a_scale, M, where)
    _vector(w_scale, N, where)
    _vector(bias, N, where)
    if out is not None:
        out_dtype = out[0]
        _need(out[1] == (M, N) and (N == 1 or out[2][1] == 1), where)
    _need(out_dtype in _FLOATS, where)
    p = bsa_linear_int8_params(M, N, K, DTYPES[out_dtype], a[2][0], w[2][0],
                               N if out is None else out[2][0])
    return device, p, ctypes.addressof(p), ((M, N), (N, 1))


def linear_int8(a, a_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None,
                dev_status=None, stream=None):
    """bsa_linear_int8: a_scale[:, None] * w_scale * (a @ w.T) + bias from int8 codes a [M, K] and
    w [N, K] (rows on 16 bytes, as ``quantize_int8`` lays them out), exact sums, fp32 or bf16 out."""
    host = _host or _load_host()
    key = (host.layout(a, a_scale, w, w_scale, bias, out), out_dtype)
    plan = _linear_plans.get(key)
    if plan is None:
        plan = _keep(_linear_plans, key, _linear_int8_plan(
            _sig(a), _sig(a_scale), _sig(w), _sig(w_scale), _sig(bias), _sig(out), out_dtype))
    device, p, ref, rows = plan
    if not _here(device, stream):
        with _elsewhere(device, stream, "linear_int8"):
            return linear_int8(a, a_scale, w, w_scale, bias, out_dtype, out, dev_status)
    if dev_status is not None:
        _need(dev_status.get_device() == device, "linear_int8")
        p = bsa_linear_int8_params.from_buffer_copy(p)
        p.dev_status = dev_status.data_ptr()
        ref = ctypes.addressof(p)
    o = host.empty(*rows, out_dtype, a) if out is None else out
    _check(host.call(lib().addresses["bsa_linear_int8"], ref, a, a_scale, w, w_scale, bias, o,
                     _raw_stream(device)), "bsa_linear_int8")
    return o


def forward_block(x, w_qkv, s_qkv, w_out, s_out, positions, freqs, top_k, gate=None, scale=None,
                  shift=None, b_qkv=None, b_out=None, pre="rms", pre_weight=None, pre_bias=None,
                  post="none", post_weight=None, post_bias=None, q_weight=None, k_weight=None,
                  layout="half", axis_pairs=None, rope_scale=1.0, eps=1e-6, qk_eps=1e-6,
                  residual_scale=1.0, branch_scale=1.0, prefix=0, variant="anchor", out=None,
                  ws=None, dev_status=None, stream=None):
    """bsa_forward_block: the attention half of a block on token rows x [B, N, C] (contiguous).

    w_qkv [3 H 128, C] and w_out [C, H 128] are int8 codes with one scale a row, as
    ``quantize_int8`` makes them; the vectors are those of ``gate_norm`` and ``rotary``.  ``out`` may
    be x.  Returns out."""
    where = "forward_block"
    vectors = (pre_weight, pre_bias, post_weight, post_bias)
    sigs = [_sig(t) for t in (w_qkv, s_qkv, w_out, s_out, positions, freqs, gate, scale, shift,
                              b_qkv, b_out, *vectors, q_weight, k_weight, out, ws, dev_status)]
    device = _one_device(where, _sig(x), *sigs)
    _need(x.dim() == 3 and x.dtype in _FLOATS and x.is_contiguous(), where)
    B, N, C = x.shape
    for w in (w_qkv, w_out):
        _need(w.dim() == 2 and w.dtype == torch.int8 and w.stride(1) == 1, where)
    H = w_out.shape[1] // 128
    _need(H >= 1 and w_qkv.shape == (3 * H * 128, C) and w_out.shape == (C, H * 128), where)
    for t, n in ((s_qkv, 3 * H * 128), (s_out, C)):
        _need(t is not None, where)
        _vector(_sig(t), n, where)
    for t, n in ((b_qkv, 3 * H * 128), (b_out, C), *((v, C) for v in vectors), (q_weight, 128),
                 (k_weight, 128)):
        _vector(_sig(t), n, where)
    pairs = [freqs.numel()] if axis_pairs is None else list(axis_pairs)
    _need(freqs.dtype == torch.float64 and freqs.is_contiguous() and freqs.dim() == 1
          and 1 <= len(pairs) <= 4 and sum(pairs) == freqs.numel(), where)
    pos = positions[:, None] if positions.dim() == 1 else positions
    _need(pos.dtype == torch.int32 and pos.dim() in (2, 3) and pos.shape[-2:] == (N, len(pairs))
          and (len(pairs) == 1 or pos.stride(-1) == 1)
          and (pos.dim() == 2 or pos.shape[0] in (1, B)), where)
    mods = [t.dtype for t in (gate, scale, shift) if t is not None]
    _need(all(d in _FLOATS and d == mods[0] for d in mods), where)
    _need(pre in NORMS and post in NORMS, where)
    _need(out is None or (out.shape == x.shape and out.dtype == x.dtype and out.is_contiguous()),
          where)
    if not _here(device, stream):
        with _elsewhere(device, stream, where):
            return forward_block(x, w_qkv, s_qkv, w_out, s_out, positions, freqs, top_k, gate,
                                 scale, shift, b_qkv, b_out, pre, pre_weight, pre_bias, post,
                                 post_weight, post_bias, q_weight, k_weight, layout, axis_pairs,
                                 rope_scale, eps, qk_eps, residual_scale, branch_scale, prefix,
                                 variant, out, ws, dev_status)
    p = params(B, H, N, top_k, prefix, variant, dev_status=dev_status)
    bp = bsa_block_params(
        C, DTYPES[x.dtype], DTYPES[mods[0]] if mods else 1, NORMS[pre], NORMS[post], eps,
        residual_scale, branch_scale, qk_eps, rope_scale, 2 * freqs.numel(), ROPE_LAYOUTS[layout],
        len(pairs), (_i32 * 4)(*pairs), *_mod(_sig(gate), B, N, C, where),
        *_mod(_sig(scale), B, N, C, where), *_mod(_sig(shift), B, N, C, where),
        pos.stride(0) if pos.dim() == 3 and pos.shape[0] > 1 else 0, pos.stride(-2),
        w_qkv.stride(0), w_out.stride(0))
    bw = bsa_block_weights(*[_addr(t) for t in (gate, scale, shift, *vectors, w_qkv, s_qkv, b_qkv,
                                                w_out, s_out, b_out, q_weight, k_weight, pos,
                                                freqs)])
    if ws is None:
        n = lib().bsa_forward_block_workspace_bytes(ctypes.byref(p), ctypes.byref(bp))
        _need(n > 0, where)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty_like(x)
    _check(lib().bsa_forward_block(ctypes.byref(p), ctypes.byref(bp), ctypes.byref(bw), _addr(x),
                                   _addr(out), _addr(ws), ws.numel() * ws.element_size(),
                                   _raw_stream(device)), "bsa_forward_block")
    return out


# --------------------------------------------------------------- allocation helpers

def stage_buffers(B, H, N, top_k, prefix=0, variant="anchor", device="cuda"):
    """Device tensors for the intermediates of the four stages."""
    p = params(B, H, N, top_k, prefix, variant)
    nb = bsa_num_blocks(p)
    kcap = bsa_select_capacity(p)
    if nb < 0:
        raise BsaError(BSA_ERR_INVALID, "stage_buffers")
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    return dict(
        qpool=torch.empty(B, H, nb, 128, dtype=f32, device=device),
        anchor=torch.empty(B, H, 128, dtype=f32, device=device),
        kpool=torch.empty(B, H, nb, 128, dtype=f32, device=device),
        ksum=torch.empty(B, H, nb, 128, dtype=bf16, device=device),
        vsum=torch.empty(B, H, nb, 128, dtype=bf16, device=device),
        bias=torch.empty(B, H, nb, dtype=f32, device=device),
        idx=torch.empty(B, H, nb, kcap, dtype=i32, device=device),
        cnt=torch.empty(B, H, nb, dtype=i32, device=device),
    )


def workspace(p: bsa_params, device="cuda") -> torch.Tensor:
    n = bsa_workspace_bytes(p)
    if n == 0:
        raise BsaError(BSA_ERR_INVALID, "bsa_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward(Q, K, V, top_k, prefix=0, variant="anchor", return_lse=False, ws=None, stream=None):
    """O = block-sparse attention(Q, K, V), bf16 [B, H, N, 128] in and out."""
    B, H, N, D = Q.shape
    p = params(B, H, N, top_k, prefix, variant, D=D)
    O = torch.empty_like(Q)
    lse = torch.empty(B, H, N, dtype=torch.float32, device=Q.device) if return_lse else None
    if ws is None:
        ws = workspace(p, Q.device)
    bsa_forward(p, Q, K, V, O, lse, ws, stream)
    return (O, lse) if return_lse else O


def fp8_operands(p: bsa_params, device="cuda"):
    """One FP8 operand set in a fresh device buffer: (buffer, struct, views).

    ``views`` maps each field of bsa_fp8_operands to a torch view of the
    buffer with the documented shape (codes as uint8)."""
    n = bsa_fp8_operands_bytes(p)
    if n == 0:
        raise BsaError(BSA_ERR_INVALID, "bsa_fp8_operands_bytes")
    buf = torch.empty(n, dtype=torch.uint8, device=device)
    ops = bsa_fp8_operands_carve(p, buf)
    B, H, N = p.B, p.H, p.N
    nb = bsa_num_blocks(p)
    nt = -(-nb // 128)
    shapes = dict(q8=(B, H, N, 128), q_scale=(B, H, nb), k8=(B, H, N, 128), k_scale=(B, H, nb),
                  vt8=(B, H, nb, 128, 128), v_scale=(B, H, nb), ks8=(B, H, nb, 128),
                  ks_scale=(B, H, nt), vst8=(B, H, nt, 128, 128), vs_scale=(B, H, nt),
                  v_ref=(B, H))
    base = buf.data_ptr()
    views = {}
    for name, shape in shapes.items():
        off = getattr(ops, name) - base
        count = math.prod(shape)
        if name.endswith("8"):
            views[name] = buf[off:off + count].view(shape)
        else:
            views[name] = buf[off:off + 4 * count].view(torch.float32).view(shape)
    return buf, ops, views


def forward_fp8(Q, K, V, top_k, prefix=0, variant="anchor", return_lse=False, ws=None,
                stream=None):
    """bsa_forward_fp8: the same call as ``forward`` with e4m3 attention operands."""
    B, H, N, D = Q.shape
    p = params(B, H, N, top_k, prefix, variant, D=D)
    O = torch.empty_like(Q)
    lse = torch.empty(B, H, N, dtype=torch.float32, device=Q.device) if return_lse else None
    if ws is None:
        ws = torch.empty(bsa_forward_fp8_workspace_bytes(p), dtype=torch.uint8, device=Q.device)
    bsa_forward_fp8(p, Q, K, V, O, lse, ws, stream)
    return (O, lse) if return_lse else O


def forward_threshold(Q, K, V, tau, prefix=0, variant="anchor", return_lse=False, ws=None,
                      stream=None):
    """bsa_forward_threshold: block-sparse attention whose lists keep the key
    blocks at least tau standard deviations above each row's mean score."""
    B, H, N, D = Q.shape
    p = params(B, H, N, 1, prefix, variant, D=D)
    O = torch.empty_like(Q)
    lse = torch.empty(B, H, N, dtype=torch.float32, device=Q.device) if return_lse else None
    if ws is None:
        ws = torch.empty(bsa_forward_threshold_workspace_bytes(p), dtype=torch.uint8,
                         device=Q.device)
    bsa_forward_threshold(p, tau, Q, K, V, O, lse, ws, stream)
    return (O, lse) if return_lse else O


def topk_from_density(rho: float, N: int, prefix: int = 0) -> int:
    """Key-block ratio -> integer top_k = ceil(rho * nbv) (the caller's conversion)."""
    nbv = -(-N // 128) - prefix // 128
    return max(1, math.ceil(rho * nbv - 1e-9))
