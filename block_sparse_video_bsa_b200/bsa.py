"""Thin ctypes binding over libbsa.so (include/bsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch tensors (device memory + streams); the functions
keep the C names.  There is no fallback: if libbsa.so is missing or the
device is not sm_100 the call raises.
"""

from __future__ import annotations

import ctypes
import math
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
                                       "shift_n")])


class bsa_gate_norm_inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "y", "gate", "scale", "shift", "post_weight",
                                               "post_bias", "pre_weight", "pre_bias")]


class bsa_quantize_int8_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "N", "S", "L", "x_dtype")]
                + [(n, _i64) for n in ("x_b", "x_n", "x_s", "ld")])


class bsa_linear_int8_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("M", "N", "K", "out_dtype")]
                + [(n, _i64) for n in ("lda", "ldw", "ldo")] + [("dev_status", ctypes.c_void_p)])


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
_SIGS["bsa_gate_norm"] = (ctypes.c_int, [ctypes.POINTER(bsa_gate_norm_params),
                                         ctypes.POINTER(bsa_gate_norm_inputs)] + [_vp] * 4)
_SIGS["bsa_quantize_int8"] = (ctypes.c_int, [ctypes.POINTER(bsa_quantize_int8_params)] + [_vp] * 4)
_SIGS["bsa_linear_int8"] = (ctypes.c_int, [ctypes.POINTER(bsa_linear_int8_params)] + [_vp] * 7)
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

def _need(ok, where):
    if not ok:
        raise BsaError(BSA_ERR_INVALID, where)


def _run(ref, stream, where, call):
    """call(stream pointer) with ref's device current; its outputs belong to the stream."""
    if stream is None:
        if ref.device.index == torch.cuda.current_device():
            return call(_stream())
        with torch.cuda.device(ref.device):
            return call(_stream())
    _need(stream.device == ref.device, where)
    with torch.cuda.stream(stream):
        return call(_stream(stream))


def _same_device(where, ref, *tensors):
    _need(ref.is_cuda, where)
    for t in tensors:
        _need(t is None or t.device == ref.device, where)


def _vector(t, n, where):
    """An fp32 vector of n values, contiguous, or None."""
    _need(t is None or (t.dtype == torch.float32 and t.shape == (n,) and t.is_contiguous()), where)


def _addr(t):
    return None if t is None else t.data_ptr()


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


def _rotary_call(parts, weights, outs, positions, freqs, layout, axis_pairs, eps, scale, inverse,
                 stream):
    ref, o = next((x, y) for x, y in zip(parts, outs) if x is not None)
    B, H, N, D = ref.shape
    p = bsa_rotary_params(B, H, N, D, 2 * freqs.numel(), ROPE_LAYOUTS[layout], len(axis_pairs),
                          (_i32 * 4)(*axis_pairs), int(inverse), DTYPES[ref.dtype],
                          DTYPES[o.dtype], scale, eps, ref.stride(0), ref.stride(1), ref.stride(2),
                          o.stride(0), o.stride(1), o.stride(2),
                          positions.stride(0) if positions.dim() == 3 and positions.shape[0] > 1
                          else 0, positions.stride(-2))
    _check(lib().bsa_rotary(ctypes.byref(p), *[_addr(x) for x in parts], _addr(positions),
                            _addr(freqs), *[_addr(w) for w in weights], *[_addr(y) for y in outs],
                            stream), "bsa_rotary")


def rotary(q, k, v, positions, freqs, layout="half", axis_pairs=None, q_weight=None, k_weight=None,
           eps=1e-6, scale=1.0, inverse=False, out=None, out_dtype=None, stream=None):
    """bsa_rotary: (Q, K, V) as [B, H, N, 128] from q, k, v viewed as [B, H, N, 128] with any
    strides (token-major projections: ``qkv[:, :, 0].transpose(1, 2)`` and so on).

    Any of q, k, v may be None.  positions int32 [N, axes] or [B, N, axes] ([N] for one axis),
    freqs fp64 [pairs] from ``rotary_freqs``; axis_pairs lists the pairs of each axis.  k and v may
    have another head count than q.  ``out`` gives the outputs (a tensor may be its own output)."""
    where = "rotary"
    parts = [q, k, v]
    given = [x for x in parts if x is not None]
    _need(given, where)
    ref = given[0]
    _same_device(where, ref, *given, positions, freqs, q_weight, k_weight)
    B, N, axis_pairs = ref.shape[0], ref.shape[2], list(axis_pairs or [freqs.numel()])
    for x in given:
        _need(x.dim() == 4 and x.dtype in (torch.bfloat16, torch.float32) and x.shape[0] == B
              and x.shape[2] == N and x.shape[3] == 128 and x.stride(3) == 1, where)
    if positions.dim() == 1:
        positions = positions[:, None]
    _need(positions.dtype == torch.int32 and positions.dim() in (2, 3)
          and positions.shape[-2:] == (N, len(axis_pairs)) and positions.stride(-1) == 1
          and (positions.dim() == 2 or positions.shape[0] in (1, B)), where)
    _need(freqs.dtype == torch.float64 and freqs.dim() == 1 and freqs.is_contiguous()
          and len(axis_pairs) <= 4, where)
    weights = [q_weight, k_weight]
    for w in weights:
        _vector(w, 128, where)

    def call(st):
        outs = list(out) if out is not None else [
            None if x is None else torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
            for x in parts]
        _need(len(outs) == 3, where)
        for x, y in zip(parts, outs):
            _need((x is None) == (y is None), where)
            _need(y is None or (y.shape == x.shape and y.device == x.device and y.stride(3) == 1
                                and y.dtype in (torch.bfloat16, torch.float32)), where)
        # one launch for the tensors that share their layout
        kinds = {}
        for i, (x, y) in enumerate(zip(parts, outs)):
            if x is not None:
                kinds.setdefault((x.shape, x.stride(), x.dtype, y.stride(), y.dtype), []).append(i)
        for ids in kinds.values():
            pick = lambda t: [t[i] if i in ids else None for i in range(len(t))]  # noqa: E731
            _rotary_call(pick(parts), pick(weights), pick(outs), positions, freqs, layout,
                         axis_pairs, eps, scale, inverse, st)
        return tuple(outs)

    return _run(ref, stream, where, call)


def _mod(t, B, N, C, where):
    """(batch stride, token stride) of a vector [C], [B or 1, C] or [B or 1, N or 1, C]."""
    if t is None:
        return 0, 0
    _need(t.shape[-1] == C and t.stride(-1) == 1 and t.dim() <= 3, where)
    if t.dim() == 1:
        return 0, 0
    _need(t.shape[0] in (1, B) and (t.dim() == 2 or t.shape[1] in (1, N)), where)
    return (t.stride(0) if t.shape[0] > 1 else 0,
            t.stride(1) if t.dim() == 3 and t.shape[1] > 1 else 0)


def gate_norm(x, y=None, gate=None, scale=None, shift=None, pre="rms", pre_weight=None,
              pre_bias=None, post="none", post_weight=None, post_bias=None, eps=1e-6,
              residual_scale=1.0, branch_scale=1.0, quantize=False, z_dtype=torch.bfloat16,
              h_out=None, want_z=True, stream=None):
    """bsa_gate_norm: (h, z) with h = residual_scale x + branch_scale gate post(y) (x itself without
    y) and z = pre(h) (1 + scale) + shift.

    x, y [B, N, C]; gate, scale, shift [C], [B, C], [B, 1, C] or [B, N, C]; weights and biases fp32
    [C].  quantize: z is (codes [B N, C] int8, scales [B N]) for ``linear_int8``.  h_out: where h
    goes (x for an update in place).  want_z=False: z is None and only h is made."""
    where = "gate_norm"
    _same_device(where, x, y, gate, scale, shift, pre_weight, pre_bias, post_weight, post_bias,
                 h_out)
    _need(x.dim() == 3 and x.dtype in (torch.bfloat16, torch.float32) and x.stride(2) == 1, where)
    B, N, C = x.shape
    _need(y is None or (y.shape == x.shape and y.stride(2) == 1
                        and y.dtype in (torch.bfloat16, torch.float32)), where)
    _need(h_out is None or (y is not None and h_out.shape == x.shape and h_out.dtype == x.dtype
                            and h_out.stride(2) == 1), where)
    _need(z_dtype in (torch.bfloat16, torch.float32) and pre in NORMS and post in NORMS, where)
    mods = [t for t in (gate, scale, shift) if t is not None]
    mod_dtype = mods[0].dtype if mods else torch.float32
    for t in mods:
        _need(t.dtype == mod_dtype and t.dtype in (torch.bfloat16, torch.float32), where)
    for w in (pre_weight, pre_bias, post_weight, post_bias):
        _vector(w, C, where)
    gs, ss, hs = (_mod(t, B, N, C, where) for t in (gate, scale, shift))

    def call(st):
        h = h_out if h_out is not None else (
            None if y is None else torch.empty((B, N, C), dtype=x.dtype, device=x.device))
        z = zs = None
        z_b = z_n = 0
        if want_z and quantize:
            z = torch.empty((B * N, -(-C // 16) * 16), dtype=torch.int8, device=x.device)
            zs = torch.empty(B * N, dtype=torch.float32, device=x.device)
            z_n = z.stride(0)
            z_b = N * z_n
        elif want_z:
            z = torch.empty((B, N, C), dtype=z_dtype, device=x.device)
            z_b, z_n = N * C, C
        h_b, h_n = (h.stride(0), h.stride(1)) if h is not None else (0, 0)
        y_b, y_n = (y.stride(0), y.stride(1)) if y is not None else (0, 0)
        p = bsa_gate_norm_params(B, N, C, NORMS[pre], NORMS[post], DTYPES[x.dtype],
                                 DTYPES[y.dtype] if y is not None else 0, DTYPES[mod_dtype],
                                 2 if quantize else DTYPES[z_dtype], eps, residual_scale,
                                 branch_scale, x.stride(0), x.stride(1), y_b, y_n, h_b, h_n, z_b,
                                 z_n, *gs, *ss, *hs)
        i = bsa_gate_norm_inputs(*[_addr(t) for t in (x, y, gate, scale, shift, post_weight,
                                                      post_bias, pre_weight, pre_bias)])
        _check(lib().bsa_gate_norm(ctypes.byref(p), ctypes.byref(i), _addr(h), _addr(z), _addr(zs),
                                   st), "bsa_gate_norm")
        if want_z and quantize:
            z = (z[:, :C], zs)
        return (x if h is None else h), z

    return _run(x, stream, where, call)


def quantize_int8(x, stream=None):
    """bsa_quantize_int8: (codes, scales) of the rows of x [M, K] or [B, N, K], or of the token rows
    of an attention output [B, H, N, D] (H D values a token).  codes int8 [rows, K] (row stride a
    multiple of 16), scales fp32 [rows]."""
    where = "quantize_int8"
    _same_device(where, x)
    _need(x.dtype in (torch.bfloat16, torch.float32) and 2 <= x.dim() <= 4 and x.stride(-1) == 1,
          where)
    if x.dim() == 4:
        (B, S, N, L), s = x.shape, (x.stride(0), x.stride(2), x.stride(1))
    elif x.dim() == 3:
        (B, N, L), S, s = x.shape, 1, (x.stride(0), x.stride(1), 0)
    else:
        B, (N, L), S, s = 1, x.shape, 1, (0, x.stride(0), 0)
    K = S * L

    def call(st):
        codes = torch.empty((B * N, -(-K // 16) * 16), dtype=torch.int8, device=x.device)
        scale = torch.empty(B * N, dtype=torch.float32, device=x.device)
        p = bsa_quantize_int8_params(B, N, S, L, DTYPES[x.dtype], *s, codes.stride(0))
        _check(lib().bsa_quantize_int8(ctypes.byref(p), _addr(x), _addr(codes), _addr(scale), st),
               "bsa_quantize_int8")
        return codes[:, :K], scale

    return _run(x, stream, where, call)


def linear_int8(a, a_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None,
                dev_status=None, stream=None):
    """bsa_linear_int8: a_scale[:, None] * w_scale * (a @ w.T) + bias from int8 codes a [M, K] and
    w [N, K] (rows on 16 bytes, as ``quantize_int8`` lays them out), exact sums, fp32 or bf16 out."""
    where = "linear_int8"
    _same_device(where, a, a_scale, w, w_scale, bias, out, dev_status)
    _need(a.dim() == 2 and w.dim() == 2 and a.dtype == w.dtype == torch.int8
          and a.stride(1) == w.stride(1) == 1 and a.shape[1] == w.shape[1], where)
    (M, K), N = a.shape, w.shape[0]
    for t, n in ((a_scale, M), (w_scale, N)):
        _need(t is not None, where)
        _vector(t, n, where)
    _vector(bias, N, where)
    _need(out is None or (out.shape == (M, N) and out.stride(1) == 1
                          and out.dtype in (torch.bfloat16, torch.float32)), where)

    def call(st):
        o = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=a.device)
        p = bsa_linear_int8_params(M, N, K, DTYPES[o.dtype], a.stride(0), w.stride(0), o.stride(0),
                                   _addr(dev_status))
        _check(lib().bsa_linear_int8(ctypes.byref(p), _addr(a), _addr(a_scale), _addr(w),
                                     _addr(w_scale), _addr(bias), _addr(o), st), "bsa_linear_int8")
        return o

    return _run(a, stream, where, call)


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
