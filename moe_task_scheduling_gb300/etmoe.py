"""Thin ctypes binding of libetmoe.so: the same entry points as include/etmoe.h.

Only argument marshalling happens here (tensors -> device pointers, the
current torch stream -> cudaStream_t).  Every step of the path runs in the
CUDA kernels of libetmoe.so.  If the library is missing, `load()` raises:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libetmoe.so")

ET_OK, ET_ERR_INVALID, ET_ERR_WORKSPACE, ET_ERR_UNSUPPORTED, ET_ERR_CUDA, ET_ERR_TIMEOUT, \
    ET_ERR_BOUNDS = range(7)

ET_SCORE_SOFTMAX, ET_SCORE_SIGMOID = range(2)

STATUS_NAMES = {0: "ET_OK", 1: "ET_ERR_INVALID", 2: "ET_ERR_WORKSPACE", 3: "ET_ERR_UNSUPPORTED",
                4: "ET_ERR_CUDA", 5: "ET_ERR_TIMEOUT", 6: "ET_ERR_BOUNDS"}


class et_opts(ctypes.Structure):
    _fields_ = [("timeout_us", ctypes.c_uint32), ("trace_cap", ctypes.c_uint32),
                ("fault_mode", ctypes.c_int32), ("fault_arg", ctypes.c_int32),
                ("trace", ctypes.c_void_p)]


class et_moe_layer_desc(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("ws_gate", ctypes.c_void_p), ("ws_up", ctypes.c_void_p),
                ("ws_down", ctypes.c_void_p), ("Fs", ctypes.c_int32), ("out", ctypes.c_void_p),
                ("x_hat", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("expert_counts", ctypes.c_void_p),
                ("perm", ctypes.c_void_p)]


class EtError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_lib = None
_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_f = ctypes.c_float
_u64 = ctypes.c_uint64

_SIGNATURES = {
    "et_version": (_i, []),
    "et_last_error_string": (ctypes.c_char_p, []),
    "et_moe_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "et_moe_layer": (_i, [_vp] * 11 + [_i, _vp] + [_i] * 5 + [_vp, _sz, _vp, _vp]),
    "et_moe_block_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "et_moe_block": (_i, [_vp, _vp, ctypes.c_float] + [_vp] * 8 + [_i] + [_vp] * 6 + [_i, _vp] +
                     [_i] * 5 + [_vp, _sz, _vp, _vp]),
    "et_moe_chain_workspace_bytes": (_sz, [_i, _vp, _i, _i, _i, _i, _i]),
    "et_moe_chain": (_i, [_i, _vp, _vp, _i, _vp] + [_i] * 5 + [_vp, _sz, _vp, _vp]),
    "et_splitk_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "et_splitk_gemm": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "et_splitk_gemm_noalloc": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "et_splitk_gemm_clc": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "et_mlp_workspace_bytes": (_sz, [_i, _i, _i]),
    "et_mlp_chain": (_i, [_vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _vp,
                          _sz, _vp, _vp]),
    "et_splitk_noalloc_status": (_i, [_vp, ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32)]),
    "et_router_topk_workspace_bytes": (_sz, [_i, _i, _i]),
    "et_router_topk": (_i, [_vp] * 8 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp]),
    "et_router_topk_bwd": (_i, [_vp] * 9 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp]),
    "et_block_norm_workspace_bytes": (_sz, [_i, _i]),
    "et_block_norm": (_i, [_vp] * 4 + [_i, ctypes.c_float, _vp, ctypes.c_float, _vp, _vp, _i, _vp,
                                       _i, _i, _vp, _sz, _vp]),
    "et_block_norm_bwd": (_i, [_vp] * 4 + [_i, ctypes.c_float, _vp, ctypes.c_float] + [_vp] * 7 +
                          [_i, _vp, _i, _i, _vp, _sz, _vp]),
    "et_w4_quantize": (_i, [_vp] * 3 + [_i] * 4 + [_vp]),
    "et_w4_dequantize": (_i, [_vp] * 3 + [_i] * 4 + [_vp]),
    "et_w4_gemv_workspace_bytes": (_sz, [_i] * 4),
    "et_w4_gemv": (_i, [_vp] * 4 + [_i, _vp] + [_i] * 4 + [_vp, _sz, _vp]),
    "et_w4_experts_workspace_bytes": (_sz, [_i] * 6),
    "et_w4_experts": (_i, [_vp] * 10 + [_i, _vp] + [_i] * 6 + [_vp, _sz, _vp]),
    "et_router_groups_workspace_bytes": (_sz, [_i, _i, _i]),
    "et_router_groups": (_i, [_vp] * 3 + [_i] * 5 + [_f] + [_vp] * 6 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp]),
    "et_router_groups_bwd": (_i, [_vp, _vp, _i, _i, _f] + [_vp] * 7 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp]),
    "et_dropout_workspace_bytes": (_sz, [_i, _i]),
    "et_dropout": (_i, [_vp] * 3 + [_f, _u64, _u64, _vp, _i, _vp, _i, _i, _vp, _sz, _vp]),
    "et_layer_norm_workspace_bytes": (_sz, [_i, _i]),
    "et_layer_norm": (_i, [_vp] * 4 + [_f, _f, _u64, _u64] + [_vp] * 3 + [_i, _vp, _i, _i, _vp, _sz, _vp]),
    "et_layer_norm_bwd": (_i, [_vp] * 3 + [_f, _f, _u64, _u64] + [_vp] * 7 + [_i, _vp, _i, _i, _vp, _sz, _vp]),
    "et_i8_quantize_workspace_bytes": (_sz, [_i, _i]),
    "et_i8_quantize": (_i, [_vp] * 3 + [_i, _vp, _i, _i, _vp, _sz, _vp]),
    "et_i8_gemm_workspace_bytes": (_sz, [_i] * 3),
    "et_i8_gemm": (_i, [_vp] * 5 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp]),
    "et_i8_gemm_opts": (_i, [_vp] * 5 + [_i, _vp] + [_i] * 3 + [_vp, _sz, _vp, _vp]),
    "et_status": (_i, [_vp, _vp, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]),
    "et_reset_status": (_i, [_vp, _vp]),
}


def load(path: Optional[str] = None):
    """Open libetmoe.so (building nothing); raises if it is not there."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libetmoe.so not found at {p}: run __graft_entry__.build() first "
                           "(there is no CPU fallback for the CUDA path)")
    L = ctypes.CDLL(p)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def exported_symbols():
    return list(_SIGNATURES)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _opts(timeout_us=0, fault_mode=0, fault_arg=0, trace=None):
    if not (timeout_us or fault_mode or trace is not None):
        return None
    cap = 0 if trace is None else (trace.numel() * trace.element_size() - 32) // 32
    return ctypes.byref(et_opts(timeout_us, cap, fault_mode, fault_arg, _ptr(trace)))


def alloc_trace(records: int, device="cuda"):
    """A zeroed device buffer for `records` trace records (see et_opts.trace)."""
    import torch
    return torch.zeros(32 + 32 * records, dtype=torch.uint8, device=device)


def read_trace(buf):
    """Decode a trace buffer: list of (type, role, a, b, cta, t_begin_ns, t_end_ns).
    The records sit in per-CTA shares of the buffer; unused slots are zero."""
    import numpy as np
    raw = buf.cpu().numpy()
    cap = (raw.size - 32) // 32
    rec = raw[32:32 + 32 * cap].reshape(-1, 32)
    ints = rec[:, :16].copy().view(np.int32).reshape(-1, 4)
    ts = rec[:, 16:].copy().view(np.uint64).reshape(-1, 2)
    return [(int(i[0]) & 0xff, int(i[0]) >> 8, int(i[1]), int(i[2]), int(i[3]), int(t[0]), int(t[1]))
            for i, t in zip(ints, ts) if t[1] != 0]


def _check(rc):
    if rc != ET_OK:
        raise EtError(rc, load().et_last_error_string().decode())


def last_error() -> str:
    return load().et_last_error_string().decode()


# ------------------------------------------------------------------ workspaces

def et_moe_workspace_bytes(T_max, H, F, E, k) -> int:
    return load().et_moe_workspace_bytes(T_max, H, F, E, k)


def et_moe_block_workspace_bytes(T_max, H, F, E, k, Fs) -> int:
    return load().et_moe_block_workspace_bytes(T_max, H, F, E, k, Fs)


def et_splitk_workspace_bytes(M_max, N, K, split) -> int:
    return load().et_splitk_workspace_bytes(M_max, N, K, split)


def et_mlp_workspace_bytes(B_max, H, F) -> int:
    return load().et_mlp_workspace_bytes(B_max, H, F)


def alloc_workspace(nbytes: int, device="cuda"):
    """A zeroed, 256-byte aligned byte buffer (torch owns the memory)."""
    import torch
    if nbytes <= 0:
        raise ValueError("invalid workspace size (shape rejected by the library)")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ compute calls

def et_moe_layer(x, w_router, router_bias, w_gate, w_up, w_down, out, *, k, T=None, d_T=None,
                 T_max=None, topk_idx=None, topk_w=None, expert_counts=None, perm=None,
                 workspace, stream=None, timeout_us=0, fault_mode=0, fault_arg=0, trace=None,
                 check=True):
    H = x.shape[1]
    E = w_router.shape[1]
    F = w_gate.shape[1]
    T_max = T_max if T_max is not None else x.shape[0]
    T = T if T is not None else x.shape[0]
    rc = load().et_moe_layer(
        _ptr(x), _ptr(w_router), _ptr(router_bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
        _ptr(out), _ptr(topk_idx), _ptr(topk_w), _ptr(expert_counts), _ptr(perm), T, _ptr(d_T),
        T_max, H, F, E, k, _ptr(workspace), workspace.numel() if hasattr(workspace, "numel") else 0,
        _opts(timeout_us, fault_mode, fault_arg, trace), _stream(stream))
    if check:
        _check(rc)
    return rc


def et_moe_block(x, gamma, eps, w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                 ws_down, out, *, k, x_hat=None, T=None, d_T=None, T_max=None, topk_idx=None,
                 topk_w=None, expert_counts=None, perm=None, workspace, stream=None, timeout_us=0,
                 fault_mode=0, fault_arg=0, trace=None, check=True):
    H = x.shape[1]
    E = w_router.shape[1]
    F = w_gate.shape[1]
    Fs = 0 if ws_gate is None else ws_gate.shape[0]
    T_max = T_max if T_max is not None else x.shape[0]
    T = T if T is not None else x.shape[0]
    rc = load().et_moe_block(
        _ptr(x), _ptr(gamma), float(eps), _ptr(w_router), _ptr(router_bias), _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), Fs, _ptr(out),
        _ptr(x_hat), _ptr(topk_idx), _ptr(topk_w), _ptr(expert_counts), _ptr(perm), T, _ptr(d_T),
        T_max, H, F, E, k, _ptr(workspace), workspace.numel() if hasattr(workspace, "numel") else 0,
        _opts(timeout_us, fault_mode, fault_arg, trace), _stream(stream))
    if check:
        _check(rc)
    return rc


def layer_desc(w_router, router_bias, w_gate, w_up, w_down, out, *, gamma=None, eps=1e-5,
               ws_gate=None, ws_up=None, ws_down=None, x_hat=None, topk_idx=None, topk_w=None,
               expert_counts=None, perm=None):
    """One layer of et_moe_chain (gamma given: a fused block)."""
    return et_moe_layer_desc(
        _ptr(gamma), float(eps), _ptr(w_router), _ptr(router_bias), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down),
        0 if ws_gate is None else ws_gate.shape[0], _ptr(out), _ptr(x_hat), _ptr(topk_idx),
        _ptr(topk_w), _ptr(expert_counts), _ptr(perm))


def _desc_array(layers):
    arr = (et_moe_layer_desc * len(layers))(*layers)
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def et_moe_chain_workspace_bytes(layers, T_max, H, F, E, k) -> int:
    arr, ptr = _desc_array(layers)
    return load().et_moe_chain_workspace_bytes(len(layers), ptr, T_max, H, F, E, k)


def et_moe_chain(layers, x, *, H, F, E, k, T=None, d_T=None, T_max=None, workspace, stream=None,
                 timeout_us=0, fault_mode=0, fault_arg=0, trace=None, check=True):
    """Chained layers in one launch: layers[l + 1] reads layers[l].out."""
    T_max = T_max if T_max is not None else x.shape[0]
    T = T if T is not None else x.shape[0]
    arr, ptr = _desc_array(layers)
    rc = load().et_moe_chain(len(layers), ptr, _ptr(x), T, _ptr(d_T), T_max, H, F, E, k,
                             _ptr(workspace),
                             workspace.numel() if hasattr(workspace, "numel") else 0,
                             _opts(timeout_us, fault_mode, fault_arg, trace), _stream(stream))
    if check:
        _check(rc)
    return rc


def et_splitk_gemm(X, Wt, Y, *, split, M=None, d_M=None, M_max=None, workspace, stream=None,
                   timeout_us=0, trace=None, check=True):
    K = X.shape[1]
    N = Wt.shape[0]
    M_max = M_max if M_max is not None else X.shape[0]
    M = M if M is not None else X.shape[0]
    rc = load().et_splitk_gemm(_ptr(X), _ptr(Wt), _ptr(Y), M, _ptr(d_M), M_max, N, K, split,
                               _ptr(workspace), workspace.numel(), _opts(timeout_us, trace=trace),
                               _stream(stream))
    if check:
        _check(rc)
    return rc


def et_splitk_gemm_clc(X, Wt, Y, *, split, M=None, d_M=None, M_max=None, workspace, stream=None,
                       timeout_us=0, check=True):
    """Split-K GEMM with the Cluster Launch Control work queue (same results)."""
    K = X.shape[1]
    N = Wt.shape[0]
    M_max = M_max if M_max is not None else X.shape[0]
    M = M if M is not None else X.shape[0]
    rc = load().et_splitk_gemm_clc(_ptr(X), _ptr(Wt), _ptr(Y), M, _ptr(d_M), M_max, N, K, split,
                                   _ptr(workspace), workspace.numel(), _opts(timeout_us),
                                   _stream(stream))
    if check:
        _check(rc)
    return rc


def et_splitk_gemm_noalloc(X, Wt, Y, *, split, M=None, stream=None, check=True):
    """Split-K GEMM with the library's built-in scratch (no workspace, no allocation)."""
    K = X.shape[1]
    N = Wt.shape[0]
    M = M if M is not None else X.shape[0]
    rc = load().et_splitk_gemm_noalloc(_ptr(X), _ptr(Wt), _ptr(Y), M, N, K, split, _stream(stream))
    if check:
        _check(rc)
    return rc


def et_splitk_noalloc_status(stream=None):
    """(code, detail) of the last no-alloc split-K call on this device (synchronises)."""
    code = ctypes.c_int32(0)
    detail = ctypes.c_int32(0)
    _check(load().et_splitk_noalloc_status(_stream(stream), ctypes.byref(code),
                                           ctypes.byref(detail)))
    return code.value, detail.value


def et_mlp_chain(x, gamma, eps, w_gate, w_up, w_down, out, *, B=None, d_B=None, B_max=None,
                 workspace, stream=None, timeout_us=0, fault_mode=0, fault_arg=0, trace=None,
                 check=True):
    H = x.shape[1]
    F = w_gate.shape[0]
    B_max = B_max if B_max is not None else x.shape[0]
    B = B if B is not None else x.shape[0]
    rc = load().et_mlp_chain(_ptr(x), _ptr(gamma), float(eps), _ptr(w_gate), _ptr(w_up),
                             _ptr(w_down), _ptr(out), B, _ptr(d_B), B_max, H, F, _ptr(workspace),
                             workspace.numel(), _opts(timeout_us, fault_mode, fault_arg, trace),
                             _stream(stream))
    if check:
        _check(rc)
    return rc


# ------------------------------------------------------------------ router, norms, dropout, 4-bit and 8-bit products
#
# These calls check what the C ABI cannot see: each tensor's type, shape,
# contiguity and device (ValueError).  They run on the tensors' device, on
# `stream` or else that device's current stream.

torch = None  # imported by the first of these calls: the library opens without it


def _bind_torch():
    """Names that every call needs, and the current stream's handle without building a Stream object
    (3 us of a call that takes 8) and the current device, where this torch has them."""
    global torch, _BF16, _F32, _I32, _U8, _I8, _raw_stream, _current_device
    import torch as t
    _BF16, _F32, _I32, _U8, _I8 = t.bfloat16, t.float32, t.int32, t.uint8, t.int8
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda dev: t.cuda.current_stream(dev).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t  # last: another thread that sees it finds the rest


def _arg(t, name, dtype, shape, dev):
    """Device pointer of a contiguous CUDA tensor of this type and shape on device `dev`, or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on CUDA device {dev}, not {t.device}")


def _device_of(t, name):
    """Index of the CUDA device that holds `t`: the first step of each of these calls."""
    if torch is None:
        _bind_torch()
    dev = t.get_device()  # -1 on the CPU
    if dev >= 0:
        return dev
    raise ValueError(f"{name} must be on a CUDA device, not {t.device}")


def _workspace_args(workspace, dev):
    if workspace is None:
        raise ValueError("workspace must be given (alloc_workspace)")
    if workspace.dtype is not _U8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on CUDA device {dev}")
    return workspace.data_ptr(), workspace.numel()


# The C calls take sizes and counts as 32-bit integers, and ctypes would cut a larger one to its low half.
_INT_MAX = (1 << 31) - 1


def _fits(sizes):
    """Refuses sizes (or-ed together) of more than 31 bits, of either sign."""
    if not -_INT_MAX <= sizes <= _INT_MAX:
        raise ValueError("sizes must be below 2^31")


def _rows(n, n_max):
    """The host's count of rows: all of them where it is not given."""
    if n is None:
        return n_max
    if not -_INT_MAX <= n <= _INT_MAX:
        raise ValueError(f"a count of rows must be in [0, {n_max}], not {n}")
    return n


def _workspace_bytes(fn, *sizes):
    return fn(*sizes) if max(sizes) <= _INT_MAX and min(sizes) >= 0 else 0


def _count_arg(d_n, dev):
    if d_n is None or isinstance(d_n, int):
        return d_n
    if d_n.dtype is not _I32 or d_n.numel() != 1 or d_n.get_device() != dev:
        raise ValueError(f"a device count must be one int32 on CUDA device {dev}")
    return d_n.data_ptr()


def _call(fn, dev, stream, args, check):
    """fn(*args, stream) with device `dev` current."""
    st = _raw_stream(dev) if stream is None else _stream(stream)
    if dev == _current_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if check and rc != ET_OK:
        _check(rc)
    return rc


@functools.lru_cache(maxsize=None)
def et_router_topk_workspace_bytes(T_max, E, k) -> int:
    return _workspace_bytes(load().et_router_topk_workspace_bytes, T_max, E, k)


def et_router_topk(logits, topk_idx, topk_w, *, token_mask=None, expert_counts=None, n_routed=None,
                   mean_prob=None, losses=None, T=None, d_T=None, workspace, stream=None, check=True):
    """Top-k of logits [T_max, E]: indices, gate weights, counts; losses[0] balance, losses[1] z."""
    dev = _device_of(logits, "logits")
    T_max, E = logits.shape
    k = topk_idx.shape[-1]
    _fits(T_max | E | k)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_router_topk, dev, stream, (
        _arg(logits, "logits", _F32, (T_max, E), dev), _arg(token_mask, "token_mask", _U8, (T_max,), dev),
        _arg(topk_idx, "topk_idx", _I32, (T_max, k), dev), _arg(topk_w, "topk_w", _F32, (T_max, k), dev),
        _arg(expert_counts, "expert_counts", _I32, (E,), dev), _arg(n_routed, "n_routed", _I32, (1,), dev),
        _arg(mean_prob, "mean_prob", _F32, (E,), dev), _arg(losses, "losses", _F32, (2,), dev),
        _rows(T, T_max), _count_arg(d_T, dev), T_max, E, k, ws, wsb), check)


def et_router_topk_bwd(logits, topk_idx, topk_w, expert_counts, n_routed, d_logits, *, token_mask=None,
                       d_losses=None, d_topk_w=None, T=None, d_T=None, workspace, stream=None, check=True):
    """Gradient of et_router_topk's losses (d_losses [2]) and gate weights (d_topk_w [T_max, k])."""
    dev = _device_of(logits, "logits")
    T_max, E = logits.shape
    k = topk_idx.shape[-1]
    _fits(T_max | E | k)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_router_topk_bwd, dev, stream, (
        _arg(logits, "logits", _F32, (T_max, E), dev), _arg(token_mask, "token_mask", _U8, (T_max,), dev),
        _arg(topk_idx, "topk_idx", _I32, (T_max, k), dev), _arg(topk_w, "topk_w", _F32, (T_max, k), dev),
        _arg(expert_counts, "expert_counts", _I32, (E,), dev), _arg(n_routed, "n_routed", _I32, (1,), dev),
        _arg(d_losses, "d_losses", _F32, (2,), dev), _arg(d_topk_w, "d_topk_w", _F32, (T_max, k), dev),
        _arg(d_logits, "d_logits", _F32, (T_max, E), dev),
        _rows(T, T_max), _count_arg(d_T, dev), T_max, E, k, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_block_norm_workspace_bytes(T_max, H) -> int:
    return _workspace_bytes(load().et_block_norm_workspace_bytes, T_max, H)


def _gate(gate, T_max, H, dev):
    """(kind, pointer, gradient's type and shape) of a gate: bf16 [H], fp32 [T_max] or bf16 [T_max, H]."""
    if gate is None:
        return 0, None, None, None
    if gate.dim() == 2:
        return 3, _arg(gate, "gate", _BF16, (T_max, H), dev), _BF16, (T_max, H)
    if gate.dtype is _F32:
        return 2, _arg(gate, "gate", _F32, (T_max,), dev), _F32, (T_max,)
    return 1, _arg(gate, "gate", _BF16, (H,), dev), _F32, (H,)


def et_block_norm(x, y, x_out, x_hat, *, gamma_post=None, gate=None, scale=1.0, gamma_pre=None, eps,
                  T=None, d_T=None, workspace, stream=None, check=True):
    """x_out = x + scale * gate * RMSNorm(y) * gamma_post and x_hat = RMSNorm(x_out) * gamma_pre."""
    dev = _device_of(x, "x")
    T_max, H = rows = x.shape
    _fits(T_max | H)
    kind, pgate, _, _ = _gate(gate, T_max, H, dev)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_block_norm, dev, stream, (
        _arg(x, "x", _BF16, rows, dev), _arg(y, "y", _BF16, rows, dev),
        _arg(gamma_post, "gamma_post", _BF16, (H,), dev), pgate, kind, scale,
        _arg(gamma_pre, "gamma_pre", _BF16, (H,), dev), eps, _arg(x_out, "x_out", _BF16, rows, dev),
        _arg(x_hat, "x_hat", _BF16, rows, dev), _rows(T, T_max), _count_arg(d_T, dev), T_max, H,
        ws, wsb), check)


def et_block_norm_bwd(x, y, d_x_out, d_x_hat, dx, dy, *, gamma_post=None, gate=None, scale=1.0, gamma_pre=None,
                      eps, d_gamma_post=None, d_gamma_pre=None, d_gate=None, T=None, d_T=None, workspace,
                      stream=None, check=True):
    """Gradient of et_block_norm: dx, dy and, where given, the parameters' (fp32; a full gate's bf16)."""
    dev = _device_of(x, "x")
    T_max, H = rows = x.shape
    _fits(T_max | H)
    kind, pgate, gdt, gsh = _gate(gate, T_max, H, dev)
    if d_gate is not None and gate is None:
        raise ValueError("d_gate needs a gate")
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_block_norm_bwd, dev, stream, (
        _arg(x, "x", _BF16, rows, dev), _arg(y, "y", _BF16, rows, dev),
        _arg(gamma_post, "gamma_post", _BF16, (H,), dev), pgate, kind, scale,
        _arg(gamma_pre, "gamma_pre", _BF16, (H,), dev), eps, _arg(d_x_out, "d_x_out", _BF16, rows, dev),
        _arg(d_x_hat, "d_x_hat", _BF16, rows, dev), _arg(dx, "dx", _BF16, rows, dev),
        _arg(dy, "dy", _BF16, rows, dev), _arg(d_gamma_post, "d_gamma_post", _F32, (H,), dev),
        _arg(d_gamma_pre, "d_gamma_pre", _F32, (H,), dev), _arg(d_gate, "d_gate", gdt, gsh, dev),
        _rows(T, T_max), _count_arg(d_T, dev), T_max, H, ws, wsb), check)


def _w4(q, scale, name, lead, N, K, dev):
    """(pointer of q, pointer of scale, group) of the 4-bit weight [*lead, N, K]."""
    shape = scale.shape
    groups = shape[-2] if len(shape) > 1 else 0
    if groups < 1 or K % groups:
        raise ValueError(f"scale of {name} must be {(*lead, 'K / group', N)} with K = {K}, not {tuple(shape)}")
    shape_q, shape_s = (*lead, N, K // 2), (*lead, groups, N)
    if q is not None and q.dtype is _U8 and scale.dtype is _BF16 and q.shape == shape_q and shape == shape_s and \
            q.is_contiguous() and scale.is_contiguous() and q.get_device() == dev == scale.get_device():
        return q.data_ptr(), scale.data_ptr(), K // groups
    return _arg(q, name, _U8, shape_q, dev), _arg(scale, f"scale of {name}", _BF16, shape_s, dev), K // groups


def _w4_convert(w, q, scale):
    dev = _device_of(w, "w")
    *lead, N, K = w.shape
    if len(lead) > 1:
        raise ValueError(f"w must be [N, K] or [E, N, K], not {tuple(w.shape)}")
    _fits(N | K | (lead[0] if lead else 1))
    pq, ps, group = _w4(q, scale, "q", lead, N, K, dev)
    return dev, _arg(w, "w", _BF16, w.shape, dev), pq, ps, (lead[0] if lead else 1, N, K, group)


def et_w4_quantize(w, q, scale, *, stream=None, check=True):
    """bf16 w [N, K] or [E, N, K] -> q uint8 [.., N, K/2] and scale bf16 [.., K/group, N]; the group
    is K / scale.shape[-2]."""
    dev, pw, pq, ps, dims = _w4_convert(w, q, scale)
    return _call(load().et_w4_quantize, dev, stream, (pw, pq, ps, *dims), check)


def et_w4_dequantize(q, scale, w, *, stream=None, check=True):
    """The bf16 values of a 4-bit weight (the inverse of et_w4_quantize's layout)."""
    dev, pw, pq, ps, dims = _w4_convert(w, q, scale)
    return _call(load().et_w4_dequantize, dev, stream, (pq, ps, pw, *dims), check)


@functools.lru_cache(maxsize=None)
def et_w4_gemv_workspace_bytes(M_max, N, K, group) -> int:
    return _workspace_bytes(load().et_w4_gemv_workspace_bytes, M_max, N, K, group)


def et_w4_gemv(X, q, scale, Y, *, M=None, d_M=None, workspace, stream=None, check=True):
    """Y = X w^T for up to 64 rows, w in 4 bits (et_w4_quantize's layout).  Beyond 32 rows et_splitk_gemm
    on the bf16 weight (et_w4_dequantize) is about as fast or faster."""
    dev = _device_of(X, "X")
    M_max, K = X.shape
    N = Y.shape[-1]
    _fits(M_max | N | K)
    pq, ps, group = _w4(q, scale, "q", (), N, K, dev)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_w4_gemv, dev, stream, (
        _arg(X, "X", _BF16, (M_max, K), dev), pq, ps, _arg(Y, "Y", _BF16, (M_max, N), dev),
        _rows(M, M_max), _count_arg(d_M, dev), M_max, N, K, group, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_w4_experts_workspace_bytes(T_max, H, F, E, k, group) -> int:
    return _workspace_bytes(load().et_w4_experts_workspace_bytes, T_max, H, F, E, k, group)


def et_w4_experts(x, topk_idx, topk_w, q_gate, s_gate, q_up, s_up, q_down, s_down, out, *, T=None, d_T=None,
                  workspace, stream=None, check=True):
    """The routed SwiGLU experts of up to 64 tokens, weights in 4 bits: gate, up [E, F, H], down [E, H, F]."""
    dev = _device_of(x, "x")
    T_max, H = x.shape
    E, F = q_gate.shape[:2]
    k = topk_idx.shape[-1]
    _fits(T_max | H | F | E | k)
    pqg, psg, group = _w4(q_gate, s_gate, "q_gate", (E,), F, H, dev)
    pqu, psu, gu = _w4(q_up, s_up, "q_up", (E,), F, H, dev)
    pqd, psd, gd = _w4(q_down, s_down, "q_down", (E,), H, F, dev)
    if not group == gu == gd:
        raise ValueError(f"gate, up and down must have one group size, not {group}, {gu}, {gd}")
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_w4_experts, dev, stream, (
        _arg(x, "x", _BF16, (T_max, H), dev), _arg(topk_idx, "topk_idx", _I32, (T_max, k), dev),
        _arg(topk_w, "topk_w", _F32, (T_max, k), dev), pqg, psg, pqu, psu, pqd, psd,
        _arg(out, "out", _BF16, (T_max, H), dev), _rows(T, T_max), _count_arg(d_T, dev), T_max, H, F, E, k,
        group, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_router_groups_workspace_bytes(T_max, E, k) -> int:
    return _workspace_bytes(load().et_router_groups_workspace_bytes, T_max, E, k)


def et_router_groups(logits, topk_idx, topk_w, *, score, n_groups=1, k_groups=1, group_best=2, bias=None, renorm=True,
                     scale=1.0, token_mask=None, expert_counts=None, n_routed=None, mean_prob=None, loss=None, T=None,
                     d_T=None, workspace, stream=None, check=True):
    """Top-k by score (ET_SCORE_SOFTMAX or ET_SCORE_SIGMOID of logits [T_max, E]) + bias within the k_groups best of
    n_groups groups: indices, gate weights, counts, balance loss."""
    dev = _device_of(logits, "logits")
    T_max, E = logits.shape
    k = topk_idx.shape[-1]
    _fits(T_max | E | k | n_groups | k_groups | group_best | score)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_router_groups, dev, stream, (
        _arg(logits, "logits", _F32, (T_max, E), dev), _arg(bias, "bias", _F32, (E,), dev),
        _arg(token_mask, "token_mask", _U8, (T_max,), dev), score, n_groups, k_groups, group_best, 1 if renorm else 0, scale,
        _arg(topk_idx, "topk_idx", _I32, (T_max, k), dev), _arg(topk_w, "topk_w", _F32, (T_max, k), dev),
        _arg(expert_counts, "expert_counts", _I32, (E,), dev), _arg(n_routed, "n_routed", _I32, (1,), dev),
        _arg(mean_prob, "mean_prob", _F32, (E,), dev), _arg(loss, "loss", _F32, (1,), dev),
        _rows(T, T_max), _count_arg(d_T, dev), T_max, E, k, ws, wsb), check)


def et_router_groups_bwd(logits, topk_idx, topk_w, expert_counts, n_routed, d_logits, *, score, renorm=True, scale=1.0,
                         token_mask=None, d_loss=None, d_topk_w=None, T=None, d_T=None, workspace, stream=None, check=True):
    """Gradient of et_router_groups's loss (d_loss [1]) and gate weights (d_topk_w [T_max, k])."""
    dev = _device_of(logits, "logits")
    T_max, E = logits.shape
    k = topk_idx.shape[-1]
    _fits(T_max | E | k | score)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_router_groups_bwd, dev, stream, (
        _arg(logits, "logits", _F32, (T_max, E), dev), _arg(token_mask, "token_mask", _U8, (T_max,), dev),
        score, 1 if renorm else 0, scale,
        _arg(topk_idx, "topk_idx", _I32, (T_max, k), dev), _arg(topk_w, "topk_w", _F32, (T_max, k), dev),
        _arg(expert_counts, "expert_counts", _I32, (E,), dev), _arg(n_routed, "n_routed", _I32, (1,), dev),
        _arg(d_loss, "d_loss", _F32, (1,), dev), _arg(d_topk_w, "d_topk_w", _F32, (T_max, k), dev),
        _arg(d_logits, "d_logits", _F32, (T_max, E), dev),
        _rows(T, T_max), _count_arg(d_T, dev), T_max, E, k, ws, wsb), check)


def _rng_args(p, seed, offset, d_rng, dev):
    """p, seed, offset and the pointer of a device {seed, offset} (int64 or uint64 [2])."""
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be in [0, 2^64)")
    if d_rng is None or isinstance(d_rng, int):
        return p, seed, offset, d_rng
    if d_rng.dtype not in (torch.int64, torch.uint64) or d_rng.shape != (2,) or not d_rng.is_contiguous() or d_rng.get_device() != dev:
        raise ValueError(f"d_rng must be two int64 or uint64 on CUDA device {dev}")
    return p, seed, offset, d_rng.data_ptr()


@functools.lru_cache(maxsize=None)
def et_dropout_workspace_bytes(T_max, H) -> int:
    return _workspace_bytes(load().et_dropout_workspace_bytes, T_max, H)


def et_dropout(x, y, out, *, p, seed=0, offset=0, d_rng=None, T=None, d_T=None, workspace, stream=None, check=True):
    """out = x + dropout(y) (x None: without it); on the gradient of out, with x None, the gradient of y."""
    dev = _device_of(y, "y")
    T_max, H = rows = y.shape
    _fits(T_max | H)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_dropout, dev, stream, (
        _arg(x, "x", _BF16, rows, dev), _arg(y, "y", _BF16, rows, dev), _arg(out, "out", _BF16, rows, dev),
        *_rng_args(p, seed, offset, d_rng, dev), _rows(T, T_max), _count_arg(d_T, dev), T_max, H, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_layer_norm_workspace_bytes(T_max, H) -> int:
    return _workspace_bytes(load().et_layer_norm_workspace_bytes, T_max, H)


def et_layer_norm(x, y, x_out, x_hat, *, gamma=None, beta=None, eps, p=0.0, seed=0, offset=0, d_rng=None, T=None, d_T=None,
                  workspace, stream=None, check=True):
    """x_out = x + dropout(y) and x_hat = LayerNorm(x_out) * gamma + beta (y, x_out, gamma, beta may be None)."""
    dev = _device_of(x, "x")
    T_max, H = rows = x.shape
    _fits(T_max | H)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_layer_norm, dev, stream, (
        _arg(x, "x", _BF16, rows, dev), _arg(y, "y", _BF16, rows, dev), _arg(gamma, "gamma", _BF16, (H,), dev),
        _arg(beta, "beta", _BF16, (H,), dev), eps, *_rng_args(p, seed, offset, d_rng, dev),
        _arg(x_out, "x_out", _BF16, rows, dev), _arg(x_hat, "x_hat", _BF16, rows, dev), _rows(T, T_max),
        _count_arg(d_T, dev), T_max, H, ws, wsb), check)


def et_layer_norm_bwd(x, y, d_x_out, d_x_hat, dx, dy, *, gamma=None, eps, p=0.0, seed=0, offset=0, d_rng=None, d_gamma=None,
                      d_beta=None, T=None, d_T=None, workspace, stream=None, check=True):
    """Gradient of et_layer_norm: dx, dy (may be None) and, where given, d_gamma and d_beta (fp32)."""
    dev = _device_of(x, "x")
    T_max, H = rows = x.shape
    _fits(T_max | H)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_layer_norm_bwd, dev, stream, (
        _arg(x, "x", _BF16, rows, dev), _arg(y, "y", _BF16, rows, dev), _arg(gamma, "gamma", _BF16, (H,), dev), eps,
        *_rng_args(p, seed, offset, d_rng, dev), _arg(d_x_out, "d_x_out", _BF16, rows, dev),
        _arg(d_x_hat, "d_x_hat", _BF16, rows, dev), _arg(dx, "dx", _BF16, rows, dev), _arg(dy, "dy", _BF16, rows, dev),
        _arg(d_gamma, "d_gamma", _F32, (H,), dev), _arg(d_beta, "d_beta", _F32, (H,), dev), _rows(T, T_max),
        _count_arg(d_T, dev), T_max, H, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_i8_quantize_workspace_bytes(M_max, K) -> int:
    return _workspace_bytes(load().et_i8_quantize_workspace_bytes, M_max, K)


def et_i8_quantize(x, q, scale, *, M=None, d_M=None, workspace, stream=None, check=True):
    """bf16 rows x [M_max, K] -> int8 q and fp32 scale [M_max], one for each row (a token, or a weight's channel)."""
    dev = _device_of(x, "x")
    M_max, K = x.shape
    _fits(M_max | K)
    ws, wsb = _workspace_args(workspace, dev)
    return _call(load().et_i8_quantize, dev, stream, (
        _arg(x, "x", _BF16, (M_max, K), dev), _arg(q, "q", _I8, (M_max, K), dev), _arg(scale, "scale", _F32, (M_max,), dev),
        _rows(M, M_max), _count_arg(d_M, dev), M_max, K, ws, wsb), check)


@functools.lru_cache(maxsize=None)
def et_i8_gemm_workspace_bytes(M_max, N, K) -> int:
    return _workspace_bytes(load().et_i8_gemm_workspace_bytes, M_max, N, K)


def et_i8_gemm(x_q, s_x, w_q, s_w, Y, *, M=None, d_M=None, workspace, stream=None, timeout_us=0, fault_mode=0, fault_arg=0,
               check=True):
    """Y = (s_x s_w^T) * (x_q w_q^T) for int8 x_q [M_max, K] and w_q [N, K] with their fp32 scales."""
    dev = _device_of(x_q, "x_q")
    M_max, K = x_q.shape
    N = Y.shape[-1]
    _fits(M_max | N | K)
    ws, wsb = _workspace_args(workspace, dev)
    args = (
        _arg(x_q, "x_q", _I8, (M_max, K), dev), _arg(s_x, "s_x", _F32, (M_max,), dev), _arg(w_q, "w_q", _I8, (N, K), dev),
        _arg(s_w, "s_w", _F32, (N,), dev), _arg(Y, "Y", _BF16, (M_max, N), dev), _rows(M, M_max), _count_arg(d_M, dev),
        M_max, N, K, ws, wsb)
    if timeout_us or fault_mode:
        return _call(load().et_i8_gemm_opts, dev, stream, (*args, _opts(timeout_us, fault_mode, fault_arg)), check)
    return _call(load().et_i8_gemm, dev, stream, args, check)


def et_status(workspace, stream=None):
    """(code, detail) of the workspace's sticky device status (synchronises)."""
    code = ctypes.c_int32(0)
    detail = ctypes.c_int32(0)
    _check(load().et_status(_ptr(workspace), _stream(stream), ctypes.byref(code),
                            ctypes.byref(detail)))
    return code.value, detail.value


def et_reset_status(workspace, stream=None):
    _check(load().et_reset_status(_ptr(workspace), _stream(stream)))
