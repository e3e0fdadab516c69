"""Thin ctypes binding of libqs_moe.so (include/qs_moe.h), same entry-point names.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (device memory supplied by PyTorch);
the stream defaults to torch's current stream.  If the library is missing this
module raises -- there is no CPU path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

from . import build as _build

QS_OK, QS_ERR_INVALID, QS_ERR_CUDA, QS_ERR_TIMEOUT, QS_ERR_UNSUPPORTED, QS_ERR_WORKSPACE = range(6)
QS_F32, QS_BF16, QS_E4M3 = 0, 1, 2

# the entry points include/qs_moe.h declares
EXPORTS = (
    "qs_status_string", "qs_abi_version", "qs_last_cuda_error", "qs_moe_workspace_bytes", "qs_workspace_init",
    "qs_read_device_status", "qs_route_topk", "qs_group_tokens", "qs_q2k_gemv_grouped", "qs_q2k_down_combine",
    "qs_shared_expert_ffn", "qs_moe_ffn", "qs_moe_ffn_launches", "qs_moe_ffn_q4k_launches", "qs_q2k_quantize",
    "qs_test_wait_timeout",
    "qs_moe_ffn_noalloc", "qs_steer_rows", "qs_moe_ffn_q4k", "qs_q4k_quantize", "qs_moe_host_workspace_bytes",
    "qs_moe_ffn_host", "qs_noalloc_read_device_status", "qs_read_routing", "qs_moe_ffn_cluster",
    "qs_rmsnorm_residual", "qs_rmsnorm_backward_workspace_bytes", "qs_rmsnorm_residual_backward", "qs_silu_mul_quant",
    "qs_fp8_matmul_workspace_bytes", "qs_fp8_matmul", "qs_dispatch_workspace_bytes", "qs_dispatch_tokens",
    "qs_combine_tokens", "qs_combine_tokens_backward",
)


class QsError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class qs_moe_shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("expert_ffn", ctypes.c_int32), ("shared_ffn", ctypes.c_int32), ("x_dtype", ctypes.c_int32)]


class qs_q2k_experts(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("expert_stride", ctypes.c_int64)]


class qs_q4k_experts(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("expert_stride", ctypes.c_int64)]


class qs_shared_expert(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("w_gate_sig", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libqs_moe.so (building it in-tree first if asked and needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"CUDA library not built: {_build.LIB} is missing (run the package build)")
    L = ctypes.CDLL(_build.LIB)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    SP = ctypes.POINTER(qs_moe_shape)
    EP = ctypes.POINTER(qs_q2k_experts)
    HP = ctypes.POINTER(qs_shared_expert)
    L.qs_status_string.restype = ctypes.c_char_p
    L.qs_status_string.argtypes = [i32]
    L.qs_abi_version.restype = i32
    L.qs_last_cuda_error.restype = i32
    L.qs_moe_workspace_bytes.restype = sz
    L.qs_moe_workspace_bytes.argtypes = [SP, i32]
    L.qs_workspace_init.argtypes = [P, sz, P]
    L.qs_read_device_status.argtypes = [P, P]
    L.qs_route_topk.argtypes = [SP, P, P, P, i32, P, P, P, sz, P]
    L.qs_group_tokens.argtypes = [SP, P, i32, P, P, P, P]
    L.qs_q2k_gemv_grouped.argtypes = [SP, P, EP, P, P, i32, P, P]
    L.qs_q2k_down_combine.argtypes = [SP, EP, P, P, P, i32, P, i32, P]
    L.qs_shared_expert_ffn.argtypes = [SP, P, HP, i32, P, i32, P, sz, P]
    L.qs_moe_ffn.argtypes = [SP, P, P, P, EP, HP, P, i32, P, sz, P]
    L.qs_moe_ffn_cluster.argtypes = [SP, P, P, P, EP, HP, P, i32, P, sz, P]
    L.qs_moe_ffn_launches.argtypes = [SP, i32, i32]
    L.qs_moe_ffn_q4k_launches.argtypes = [SP, i32, i32]
    L.qs_moe_ffn_noalloc.argtypes = [SP, P, P, P, EP, HP, P, i32, P]
    L.qs_noalloc_read_device_status.restype = i32
    L.qs_read_routing.argtypes = [SP, i32, P, sz, P, P, P]
    L.qs_noalloc_read_device_status.argtypes = [P]
    L.qs_q2k_quantize.argtypes = [P, i64, i64, P, P]
    L.qs_test_wait_timeout.argtypes = [P, sz, i32, P]
    L.qs_steer_rows.argtypes = [P, P, ctypes.c_float, i32, i32, P]
    L.qs_moe_ffn_q4k.argtypes = [SP, P, P, P, ctypes.POINTER(qs_q4k_experts), HP, P, i32, P, sz, P]
    L.qs_q4k_quantize.argtypes = [P, i64, i64, P, P]
    L.qs_moe_host_workspace_bytes.restype = sz
    L.qs_moe_host_workspace_bytes.argtypes = [SP, i32]
    L.qs_moe_ffn_host.argtypes = [SP, P, P, P, EP, HP, P, i32, P, sz, P]
    # the row operators take one packed struct each: a call of twenty ctypes arguments costs 1.3 us more than one
    for name in ("qs_rmsnorm_residual", "qs_rmsnorm_residual_backward", "qs_silu_mul_quant", "qs_fp8_matmul",
                 "qs_dispatch_tokens", "qs_combine_tokens", "qs_combine_tokens_backward"):
        getattr(L, name).argtypes = [ctypes.c_char_p, P]
    L.qs_rmsnorm_backward_workspace_bytes.argtypes = [i32]
    L.qs_fp8_matmul_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.qs_dispatch_workspace_bytes.argtypes = [i32, i32, i32]
    for name in ("qs_rmsnorm_backward_workspace_bytes", "qs_fp8_matmul_workspace_bytes", "qs_dispatch_workspace_bytes"):
        getattr(L, name).restype = sz
    for name in EXPORTS:
        if name not in ("qs_status_string", "qs_abi_version", "qs_last_cuda_error", "qs_moe_workspace_bytes",
                        "qs_moe_host_workspace_bytes", "qs_rmsnorm_backward_workspace_bytes",
                        "qs_fp8_matmul_workspace_bytes", "qs_dispatch_workspace_bytes"):
            getattr(L, name).restype = i32
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().qs_status_string(code).decode()


def _dptr(t):
    """Address of a contiguous CUDA tensor; None and raw integer addresses pass through."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"expected a tensor in device memory, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _hptr(t):
    """Address of a contiguous host tensor (pinned, for asynchronous copies)."""
    if t is None or isinstance(t, int):
        return t
    if t.is_cuda:
        raise ValueError("expected a tensor in host memory, got one on the device")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream().cuda_stream without the Stream object, a third of a call's host time
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need_rows(t, n_tokens, row_bytes, what):
    """Reject a tensor smaller than n_tokens rows of row_bytes (a raw address is taken as given)."""
    if t is None or isinstance(t, int):
        return
    have = t.numel() * t.element_size()
    if have < n_tokens * row_bytes:
        raise ValueError(f"{what}: {have} bytes, need {n_tokens} rows of {row_bytes} bytes")


def _layer_io(shape, x, out, n_tokens):
    _need_rows(x, n_tokens, shape.hidden * (2 if shape.x_dtype == QS_BF16 else 4), "x")
    _need_rows(out, n_tokens, shape.hidden * 4, "out")


def _check(rc: int, what: str):
    if rc != QS_OK:
        raise QsError(rc, what)


def make_shape(hidden, n_experts, top_k, expert_ffn, shared_ffn, x_dtype) -> qs_moe_shape:
    return qs_moe_shape(hidden, n_experts, top_k, expert_ffn, shared_ffn, x_dtype)


def make_experts(blocks, expert_stride: int) -> qs_q2k_experts:
    return qs_q2k_experts(_dptr(blocks), expert_stride)


def make_q4k_experts(blocks, expert_stride: int) -> qs_q4k_experts:
    return qs_q4k_experts(_dptr(blocks), expert_stride)


def make_shared(w_gate, w_up, w_down, w_gate_sig) -> qs_shared_expert:
    return qs_shared_expert(_dptr(w_gate), _dptr(w_up), _dptr(w_down), _dptr(w_gate_sig))


# ------------------------------------------------------------------ entry points

def qs_abi_version() -> int:
    return load().qs_abi_version()


def qs_last_cuda_error() -> int:
    return load().qs_last_cuda_error()


def qs_moe_workspace_bytes(shape: qs_moe_shape, max_tokens: int) -> int:
    return load().qs_moe_workspace_bytes(ctypes.byref(shape), max_tokens)


def qs_workspace_init(workspace, stream=None):
    _check(load().qs_workspace_init(_dptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "qs_workspace_init")


def qs_read_device_status(workspace, stream=None) -> int:
    return load().qs_read_device_status(_dptr(workspace), _stream(stream))


def qs_route_topk(shape, x, router_w, router_bias, n_tokens, topk_ids, topk_w, workspace, stream=None):
    _check(load().qs_route_topk(ctypes.byref(shape), _dptr(x), _dptr(router_w), _dptr(router_bias), n_tokens,
                                _dptr(topk_ids), _dptr(topk_w), _dptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)), "qs_route_topk")


def qs_group_tokens(shape, topk_ids, n_tokens, counts, offsets, perm, stream=None):
    _check(load().qs_group_tokens(ctypes.byref(shape), _dptr(topk_ids), n_tokens, _dptr(counts), _dptr(offsets),
                                  _dptr(perm), _stream(stream)), "qs_group_tokens")


def qs_q2k_gemv_grouped(shape, x, experts: qs_q2k_experts, offsets, perm, n_tokens, h_out, stream=None):
    _check(load().qs_q2k_gemv_grouped(ctypes.byref(shape), _dptr(x), ctypes.byref(experts), _dptr(offsets),
                                      _dptr(perm), n_tokens, _dptr(h_out), _stream(stream)), "qs_q2k_gemv_grouped")


def qs_q2k_down_combine(shape, experts: qs_q2k_experts, h, topk_ids, topk_w, n_tokens, out, accumulate=False,
                        stream=None):
    _check(load().qs_q2k_down_combine(ctypes.byref(shape), ctypes.byref(experts), _dptr(h), _dptr(topk_ids),
                                      _dptr(topk_w), n_tokens, _dptr(out), int(bool(accumulate)), _stream(stream)),
           "qs_q2k_down_combine")


def qs_shared_expert_ffn(shape, x, shared: qs_shared_expert, n_tokens, out, workspace, accumulate=False,
                         stream=None):
    _check(load().qs_shared_expert_ffn(ctypes.byref(shape), _dptr(x), ctypes.byref(shared), n_tokens, _dptr(out),
                                       int(bool(accumulate)), _dptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)),
           "qs_shared_expert_ffn")


def qs_moe_ffn(shape, x, router_w, router_bias, experts: qs_q2k_experts, shared, out, n_tokens, workspace,
               stream=None):
    _layer_io(shape, x, out, n_tokens)
    _check(load().qs_moe_ffn(ctypes.byref(shape), _dptr(x), _dptr(router_w), _dptr(router_bias),
                             ctypes.byref(experts), None if shared is None else ctypes.byref(shared), _dptr(out),
                             n_tokens, _dptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream)), "qs_moe_ffn")


def qs_moe_ffn_cluster(shape, x, router_w, router_bias, experts: qs_q2k_experts, shared, out, n_tokens, workspace,
                       stream=None):
    """The whole layer through the cluster decode kernel alone (QsError QS_ERR_UNSUPPORTED outside its plan)."""
    _layer_io(shape, x, out, n_tokens)
    _check(load().qs_moe_ffn_cluster(ctypes.byref(shape), _dptr(x), _dptr(router_w), _dptr(router_bias),
                                     ctypes.byref(experts), None if shared is None else ctypes.byref(shared), _dptr(out),
                                     n_tokens, _dptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "qs_moe_ffn_cluster")


def qs_moe_ffn_noalloc(shape, x, router_w, router_bias, experts: qs_q2k_experts, shared, out, n_tokens,
                       stream=None):
    """The whole layer with its scratch in a fixed array inside the library (no workspace argument)."""
    _layer_io(shape, x, out, n_tokens)
    _check(load().qs_moe_ffn_noalloc(ctypes.byref(shape), _dptr(x), _dptr(router_w), _dptr(router_bias),
                                     ctypes.byref(experts), None if shared is None else ctypes.byref(shared),
                                     _dptr(out), n_tokens, _stream(stream)), "qs_moe_ffn_noalloc")


def qs_read_routing(shape, n_tokens, workspace, stream=None):
    """(ids int32 [n_tokens, k], weights fp32 [n_tokens, k]) the last qs_moe_ffn call on workspace used."""
    k = shape.top_k
    ids = np.zeros((n_tokens, k), np.int32)
    w = np.zeros((n_tokens, k), np.float32)
    _check(load().qs_read_routing(ctypes.byref(shape), n_tokens, _dptr(workspace),
                                  workspace.numel() * workspace.element_size(), ids.ctypes.data, w.ctypes.data,
                                  _stream(stream)), "qs_read_routing")
    return ids, w


def qs_noalloc_read_device_status(stream=None) -> int:
    """Sticky device status of the qs_moe_ffn_noalloc array on the current device, cleared by the read."""
    return load().qs_noalloc_read_device_status(_stream(stream))


def qs_steer_rows(out, direction, scale, n_tokens, stream=None):
    """In place, per row of out [n_tokens, hidden] fp32: y <- y - scale * direction * (direction . y)."""
    _check(load().qs_steer_rows(_dptr(out), _dptr(direction), float(scale), n_tokens, out.shape[-1],
                                _stream(stream)), "qs_steer_rows")


def qs_moe_ffn_host(shape, x_host, router_w, router_bias, experts: qs_q2k_experts, shared, out_host, n_tokens,
                    workspace, stream=None):
    """The whole layer with x_host and out_host in (pinned) host memory; copies are queued on the stream."""
    _layer_io(shape, x_host, out_host, n_tokens)
    _check(load().qs_moe_ffn_host(ctypes.byref(shape), _hptr(x_host), _dptr(router_w), _dptr(router_bias),
                                  ctypes.byref(experts), None if shared is None else ctypes.byref(shared),
                                  _hptr(out_host), n_tokens, _dptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "qs_moe_ffn_host")


def alloc_host_workspace(shape: qs_moe_shape, max_tokens: int, device="cuda"):
    """A zero-initialised workspace for qs_moe_ffn_host."""
    n = load().qs_moe_host_workspace_bytes(ctypes.byref(shape), max_tokens)
    if n == 0:
        raise QsError(QS_ERR_INVALID, "qs_moe_host_workspace_bytes")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def qs_moe_ffn_launches(shape, n_tokens, has_shared=True) -> int:
    return load().qs_moe_ffn_launches(ctypes.byref(shape), n_tokens, int(bool(has_shared)))


def qs_moe_ffn_q4k_launches(shape, n_tokens, has_shared=True) -> int:
    return load().qs_moe_ffn_q4k_launches(ctypes.byref(shape), n_tokens, int(bool(has_shared)))


def qs_q2k_quantize(w, out, stream=None):
    rows, K = w.shape
    _check(load().qs_q2k_quantize(_dptr(w), rows, K, _dptr(out), _stream(stream)), "qs_q2k_quantize")


def qs_q4k_quantize(w, out, stream=None):
    rows, K = w.shape
    _check(load().qs_q4k_quantize(_dptr(w), rows, K, _dptr(out), _stream(stream)), "qs_q4k_quantize")


def qs_moe_ffn_q4k(shape, x, router_w, router_bias, experts: qs_q4k_experts, shared, out, n_tokens, workspace,
                   stream=None):
    """The whole layer with Q4_K routed experts (same arguments as qs_moe_ffn)."""
    _layer_io(shape, x, out, n_tokens)
    _check(load().qs_moe_ffn_q4k(ctypes.byref(shape), _dptr(x), _dptr(router_w), _dptr(router_bias),
                                 ctypes.byref(experts), None if shared is None else ctypes.byref(shared), _dptr(out),
                                 n_tokens, _dptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "qs_moe_ffn_q4k")


def qs_test_wait_timeout(workspace, limit_us, stream=None):
    _check(load().qs_test_wait_timeout(_dptr(workspace), workspace.numel() * workspace.element_size(), limit_us,
                                       _stream(stream)), "qs_test_wait_timeout")


# ------------------------------------------------------------------ row operators
#
# Matrices are 2-D tensors whose columns are contiguous; rows may be strided.  fp32 and bf16 tensors are
# torch.float32 and torch.bfloat16, e4m3 codes torch.float8_e4m3fn.  All of a call's tensors are on the current device.

_WIDE = {torch.float32: QS_F32, torch.bfloat16: QS_BF16}
_E4M3 = {torch.float8_e4m3fn: QS_E4M3}

# the argument structs of include/qs_moe.h, as they lie in memory
_ROWS, _CODES = "Pqi4x", "PqPq"
ARGS = {
    "qs_rmsnorm_residual": struct.Struct("@" + 4 * _ROWS + _CODES + "Pfii4x"),
    "qs_rmsnorm_residual_backward": struct.Struct("@" + 4 * _ROWS + "PPPNfii4x"),
    "qs_silu_mul_quant": struct.Struct("@" + _ROWS + _CODES + "Pii"),
    "qs_fp8_matmul": struct.Struct("@" + _CODES + "PqqPP" + _ROWS + "PNiiii"),
    "qs_dispatch_tokens": struct.Struct("@PPPPP" + 2 * _ROWS + "PqPqPNiiii"),
    "qs_combine_tokens": struct.Struct("@" + 2 * _ROWS + "PPiii4x"),
    "qs_combine_tokens_backward": struct.Struct("@" + 3 * _ROWS + "PPPiii4x"),
}
_pack_norm, _pack_norm_bwd, _pack_silu, _pack_matmul, _pack_dispatch, _pack_combine, _pack_combine_bwd = (
    a.pack for a in ARGS.values())


_F32 = {torch.float32: QS_F32}
_I32 = {torch.int32: 0}
_current_device = torch._C._cuda_getDevice


def _refuse(t, what, shape, dtypes, dev):
    """Say what is wrong with a tensor that _matrix or _flat does not take."""
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a tensor in device memory, got one on {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, the call's first operand on cuda:{dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: {t.dtype} is not one of {', '.join(str(d) for d in dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{what}: expected contiguous {'columns' if t.dim() > 1 else 'elements'}")


def _device(t, what):
    """The device of a call's first operand.  The library launches on the current device, so it has to be that one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: expected a tensor in device memory, got one on {t.device}")
    if dev != _current_device():
        raise ValueError(f"{what}: on cuda:{dev}, but cuda:{_current_device()} is the current device")
    return dev


def _matrix(t, what, shape, dev, dtypes=_WIDE):
    """(address, row stride, type) of a matrix of this shape on device dev."""
    kind = dtypes.get(t.dtype)
    if kind is None or t.shape != shape or t.get_device() != dev:
        _refuse(t, what, shape, dtypes, dev)
    stride, col = t.stride()
    if col != 1 and shape[1] > 1 and shape[0] > 0:
        _refuse(t, what, shape, dtypes, dev)
    return t.data_ptr(), stride, kind


def _codes(q, scale, what, shape, dev):
    """(codes, stride, scales, stride) of an e4m3 matrix."""
    if scale is None:
        raise ValueError(f"{what}: e4m3 codes come with scales")
    a, s, _ = _matrix(q, what, shape, dev, _E4M3)
    b, u, _ = _matrix(scale, what + " scale", (shape[0], (shape[1] + 127) // 128), dev, _F32)
    return a, s, b, u


def _flat(t, what, shape, dev, dtypes=_F32):
    """Address of a contiguous tensor of this shape on device dev."""
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, what, shape, dtypes, dev)
    return t.data_ptr()


def _two(t, what):
    """The shape of a matrix."""
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a matrix, got {t.dim()} dimensions")
    return t.shape


def _ws(workspace, dev):
    """(address, bytes) of a workspace on device dev."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(workspace, "workspace", workspace.shape, (workspace.dtype,), dev)
    return workspace.data_ptr(), workspace.nbytes


def _stream_of(dev, stream):
    """The given stream, or the current one of the device."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def qs_rmsnorm_residual(x, residual, weight, eps, sum_out=None, y=None, q=None, q_scale=None, stream=None):
    """Per row: s = x + residual (residual may be None), v = s * weight / sqrt(mean(s^2) + eps); sum_out gets s,
    y gets v, q and q_scale get v as e4m3 codes with a scale per 128 columns (each may be None)."""
    shape = _two(x, "x")
    dev = _device(x, "x")
    xp, xs, xt = _matrix(x, "x", shape, dev)
    rp, rs, rt = (0, 0, 0) if residual is None else _matrix(residual, "residual", shape, dev)
    sp, ss, st = (0, 0, 0) if sum_out is None else _matrix(sum_out, "sum_out", shape, dev)
    yp, ys, yt = (0, 0, 0) if y is None else _matrix(y, "y", shape, dev)
    qp, qs, qsp, qss = (0, 0, 0, 0) if q is None and q_scale is None else _codes(q, q_scale, "q", shape, dev)
    rc = (_lib or load()).qs_rmsnorm_residual(
        _pack_norm(xp, xs, xt, rp, rs, rt, sp, ss, st, yp, ys, yt, qp, qs, qsp, qss, _flat(weight, "weight", shape[1:], dev), eps,
                   shape[0], shape[1]), _stream_of(dev, stream))
    if rc:
        raise QsError(rc, "qs_rmsnorm_residual")


def alloc_rmsnorm_backward_workspace(hidden, device="cuda"):
    """A workspace for qs_rmsnorm_residual_backward."""
    return _alloc(load().qs_rmsnorm_backward_workspace_bytes(hidden), "qs_rmsnorm_backward_workspace_bytes", device)


def qs_rmsnorm_residual_backward(sum, weight, eps, dy, dsum, dx, dweight=None, workspace=None, stream=None):
    """dx, the gradient of x and of residual alike, and dweight (None: left out) from dy and dsum (None: no gradient
    by the residual stream); sum is what qs_rmsnorm_residual stored in sum_out."""
    shape = _two(sum, "sum")
    if dweight is not None and workspace is None:
        raise ValueError("dweight needs a workspace")
    dev = _device(sum, "sum")
    rc = (_lib or load()).qs_rmsnorm_residual_backward(
        _pack_norm_bwd(*_matrix(sum, "sum", shape, dev), *_matrix(dy, "dy", shape, dev),
                       *((0, 0, 0) if dsum is None else _matrix(dsum, "dsum", shape, dev)), *_matrix(dx, "dx", shape, dev),
                       _flat(weight, "weight", shape[1:], dev), 0 if dweight is None else _flat(dweight, "dweight", shape[1:], dev),
                       *((0, 0) if workspace is None else _ws(workspace, dev)), eps, *shape), _stream_of(dev, stream))
    _check(rc, "qs_rmsnorm_residual_backward")


def qs_silu_mul_quant(gate_up, q, q_scale, n_rows=None, stream=None):
    """q, q_scale [rows, F]: silu(gate) * up of gate_up [rows, 2F] as e4m3 codes with scales; n_rows (an int32 tensor
    on the device, or None): rows at and beyond its first element are left alone."""
    shape = _two(q, "q")
    rows, ffn = shape
    dev = _device(q, "q")
    gp, gs, gt = _matrix(gate_up, "gate_up", (rows, 2 * ffn), dev)
    qp, qs, qsp, qss = _codes(q, q_scale, "q", shape, dev)
    if n_rows is not None and n_rows.numel() == 0:  # its address is 0, which means no limit
        raise ValueError("n_rows: expected an element")
    rc = (_lib or load()).qs_silu_mul_quant(
        _pack_silu(gp, gs, gt, qp, qs, qsp, qss, 0 if n_rows is None else _flat(n_rows, "n_rows", n_rows.shape, dev, _I32), rows, ffn),
        _stream_of(dev, stream))
    if rc:
        raise QsError(rc, "qs_silu_mul_quant")


def alloc_fp8_matmul_workspace(n_rows, n_cols, n_inner, n_experts=1, device="cuda"):
    """A zero-initialised workspace for qs_fp8_matmul of up to this size."""
    return _alloc(load().qs_fp8_matmul_workspace_bytes(n_rows, n_cols, n_inner, n_experts), "qs_fp8_matmul_workspace_bytes", device)


def qs_fp8_matmul(a, a_scale, w, w_scale, out, workspace, offsets=None, stream=None):
    """out [rows, N] = a [rows, K] times w [N, K] (or, with offsets int32 [E + 1], w [E, N, K] of the expert whose
    rows offsets[e] .. offsets[e + 1] - 1 are) transposed; e4m3 codes, rows of both at 16-byte boundaries, with a scale per
    row and 128 columns of a and per 128 x 128 block of w."""
    shape = _two(a, "a")
    rows, inner = shape
    if offsets is not None and w.dim() != 3:
        raise ValueError(f"w: expected [experts, cols, inner], got {w.dim()} dimensions")
    dev = _device(a, "a")
    if offsets is None:
        experts, cols, off, expert_stride = 1, _two(w, "w")[0], 0, 0
        wp, w_stride, _ = _matrix(w, "w", (cols, inner), dev, _E4M3)
        blocks = ((cols + 127) // 128, (inner + 127) // 128)
    else:
        experts, cols, k = w.shape
        if w.dtype not in _E4M3 or k != inner or w.get_device() != dev or (w.stride(2) != 1 and inner > 1):
            _refuse(w, "w", (experts, cols, inner), _E4M3, dev)
        wp = w.data_ptr()
        expert_stride, w_stride, _ = w.stride()
        blocks = (experts, (cols + 127) // 128, (inner + 127) // 128)
        off = _flat(offsets, "offsets", (experts + 1,), dev, _I32)
    ap, as_, sp, ss = _codes(a, a_scale, "a", shape, dev)
    op, os_, ot = _matrix(out, "out", (rows, cols), dev)
    ws, ws_bytes = _ws(workspace, dev)
    rc = (_lib or load()).qs_fp8_matmul(
        _pack_matmul(ap, as_, sp, ss, wp, w_stride, expert_stride, _flat(w_scale, "w scale", blocks, dev), off, op, os_, ot, ws, ws_bytes,
                     experts, rows, cols, inner), _stream_of(dev, stream))
    if rc:
        raise QsError(rc, "qs_fp8_matmul")


def alloc_dispatch_workspace(n_tokens, top_k, n_experts, device="cuda"):
    """A workspace for qs_dispatch_tokens of up to this size."""
    return _alloc(load().qs_dispatch_workspace_bytes(n_tokens, top_k, n_experts), "qs_dispatch_workspace_bytes", device)


def qs_dispatch_tokens(topk_ids, x, x_scale, counts, offsets, perm, pos, xs, xs_scale, workspace, stream=None):
    """The plan of topk_ids [tokens, k] (counts [E], offsets [E + 1], perm [tokens * k], pos [tokens, k], all int32)
    and xs [tokens * k, hidden], the rows of x sorted by expert; x e4m3 brings x_scale along to xs_scale.  x and xs
    None: the plan alone."""
    shape = _two(topk_ids, "topk_ids")
    tokens, k = shape
    n, experts, hidden = tokens * k, counts.numel(), 0
    xp = xs_ = xt = yp = ys = sp = ss = tp = ts = 0
    if (x is None) != (xs is None):
        raise ValueError("x and xs come together")
    dev = _device(topk_ids, "topk_ids")
    if x is not None:
        hidden = _two(x, "x")[1]
        if x.dtype is torch.float8_e4m3fn:
            xp, xs_, sp, ss = _codes(x, x_scale, "x", (tokens, hidden), dev)
            yp, ys, tp, ts = _codes(xs, xs_scale, "xs", (n, hidden), dev)
            xt = QS_E4M3
        else:
            xp, xs_, xt = _matrix(x, "x", (tokens, hidden), dev)
            yp, ys, _ = _matrix(xs, "xs", (n, hidden), dev, {x.dtype: xt})
    ws, ws_bytes = _ws(workspace, dev)
    rc = (_lib or load()).qs_dispatch_tokens(
        _pack_dispatch(_flat(topk_ids, "topk_ids", shape, dev, _I32), _flat(counts, "counts", (experts,), dev, _I32),
                       _flat(offsets, "offsets", (experts + 1,), dev, _I32), _flat(perm, "perm", (n,), dev, _I32), _flat(pos, "pos", shape, dev, _I32),
                       xp, xs_, xt, yp, ys, xt, sp, ss, tp, ts, ws, ws_bytes, tokens, k, experts, hidden), _stream_of(dev, stream))
    if rc:
        raise QsError(rc, "qs_dispatch_tokens")


def qs_combine_tokens(y, pos, topk_w, out, stream=None):
    """out [tokens, hidden]: the sum over a token's slots of topk_w (None: 1) times its row of y [tokens * k, hidden]."""
    shape = _two(pos, "pos")
    tokens, k = shape
    hidden = _two(out, "out")[1]
    dev = _device(pos, "pos")
    yp, ys, yt = _matrix(y, "y", (tokens * k, hidden), dev)
    op, os_, ot = _matrix(out, "out", (tokens, hidden), dev)
    rc = (_lib or load()).qs_combine_tokens(
        _pack_combine(yp, ys, yt, op, os_, ot, _flat(pos, "pos", shape, dev, _I32), 0 if topk_w is None else _flat(topk_w, "topk_w", shape, dev),
                      tokens, k, hidden), _stream_of(dev, stream))
    if rc:
        raise QsError(rc, "qs_combine_tokens")


def qs_combine_tokens_backward(dout, y, pos, topk_w, dy, dtopk_w=None, stream=None):
    """Gradient of qs_combine_tokens: dy [tokens * k, hidden] and dtopk_w [tokens, k] (None: left out; y may then be
    None)."""
    shape = _two(pos, "pos")
    tokens, k = shape
    hidden = _two(dout, "dout")[1]
    if dtopk_w is not None and y is None:
        raise ValueError("dtopk_w needs y")
    dev = _device(pos, "pos")
    rc = (_lib or load()).qs_combine_tokens_backward(
        _pack_combine_bwd(*_matrix(dout, "dout", (tokens, hidden), dev), *((0, 0, 0) if y is None else _matrix(y, "y", (tokens * k, hidden), dev)),
                          *_matrix(dy, "dy", (tokens * k, hidden), dev), _flat(pos, "pos", shape, dev, _I32),
                          0 if topk_w is None else _flat(topk_w, "topk_w", shape, dev),
                          0 if dtopk_w is None else _flat(dtopk_w, "dtopk_w", shape, dev), tokens, k, hidden), _stream_of(dev, stream))
    _check(rc, "qs_combine_tokens_backward")


def _alloc(n, what, device):
    if n == 0:
        raise QsError(QS_ERR_INVALID, what)
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


# ------------------------------------------------------------------ conveniences

def alloc_workspace(shape: qs_moe_shape, max_tokens: int, device="cuda"):
    """A zero-initialised workspace tensor (256-byte aligned by the CUDA caching allocator)."""
    n = qs_moe_workspace_bytes(shape, max_tokens)
    if n == 0:
        raise QsError(QS_ERR_INVALID, "qs_moe_workspace_bytes")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws
