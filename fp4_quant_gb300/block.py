"""The operators around a gated activation: block norms, expert routing and
linear layers (``include/glu_block.h``), as calls on torch tensors.

Like ``fwd``/``bwd``/``gemm``, these check their tensors, allocate what the
call returns (unless ``out`` holds it) and its workspace, and raise
``GluQuantError`` on a status other than 0, with nothing launched.  Matrices
are CUDA tensors on the current device with unit column stride, a row stride
that is a multiple of 8 elements and a 16-byte aligned base; widths are free
(a result whose width is not a multiple of 8 is a view of a wider buffer).  A
matrix of rows (not a weight, a gate or an ``out``) with another row stride,
such as the contiguous one of odd width that ``fwd`` returns, is copied first.
Calls go to the current stream, or to ``stream`` (a ``torch.cuda.Stream`` or a
raw handle), to which what they allocate then belongs; ordering it with the
streams of the operands is the caller's, as for any torch call.
"""
from __future__ import annotations

import ctypes

import torch

from . import (ACT_IDENTITY, FMT_BF16, FMT_FP32, GLU_OK, GluQuantError, _lib)

__all__ = ["block_norm", "block_norm_bwd", "route", "dispatch", "dispatch_bwd", "combine", "combine_bwd", "linear", "linear_bwd",
           "block_device_errors", "block_abi_version"]

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_i32, _i64, _f32, _ptr, _size = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class NormFwdArgs(ctypes.Structure):
    """Mirror of ``glu_block_norm_fwd_args``."""
    _fields_ = ([(n, _i32) for n in ("x_fmt", "w_fmt")] + [(n, _f32) for n in ("alpha", "w_offset", "eps")] + [("reserved", _i32)]
                + [(n, _i64) for n in ("M", "D", "gates", "ld_x", "ld_branch", "ld_gate", "ld_r", "ld_y")]
                + [(n, _ptr) for n in ("x", "branch", "gate", "w_pre", "w_post", "r", "y", "rstd_pre", "rstd_post")])


class NormBwdArgs(ctypes.Structure):
    """Mirror of ``glu_block_norm_bwd_args``."""
    _fields_ = ([(n, _i32) for n in ("x_fmt", "w_fmt")] + [(n, _f32) for n in ("alpha", "w_offset")]
                + [(n, _i64) for n in ("M", "D", "gates", "ld_r", "ld_branch", "ld_gate", "ld_dy", "ld_dr", "ld_dx", "ld_dbranch")]
                + [(n, _ptr) for n in ("r", "branch", "gate", "w_pre", "w_post", "rstd_pre", "rstd_post", "dy", "dr", "dx",
                                       "dbranch", "dw_pre", "dw_post", "dgate", "workspace")] + [("workspace_bytes", _size)])


class RouteArgs(ctypes.Structure):
    """Mirror of ``glu_block_route_args``."""
    _fields_ = [("id_bytes", _i32), ("E", _i32), ("T", _i64), ("K", _i64), ("ids", _ptr), ("slot", _ptr), ("src", _ptr),
                ("offsets", _ptr), ("workspace", _ptr), ("workspace_bytes", _size)]


class RowsArgs(ctypes.Structure):
    """Mirror of ``glu_block_rows_args``."""
    _fields_ = ([(n, _i64) for n in ("T", "K", "D", "ld_tokens", "ld_rows", "ld_rows_out", "ld_residual")]
                + [(n, _ptr) for n in ("slot", "src", "w", "tokens_in", "rows_in", "residual", "tokens_out", "rows_out", "dw")])


class LinearFwdArgs(ctypes.Structure):
    """Mirror of ``glu_block_linear_fwd_args``."""
    _fields_ = ([(n, _i32) for n in ("act", "b_fmt", "E", "reserved")]
                + [(n, _i64) for n in ("M", "N", "K", "ld_x", "ld_w", "stride_w", "ld_residual", "ld_y", "ld_z")]
                + [(n, _ptr) for n in ("x", "w", "bias", "residual", "offsets", "y", "z", "workspace")] + [("workspace_bytes", _size)])


class LinearBwdArgs(ctypes.Structure):
    """Mirror of ``glu_block_linear_bwd_args``."""
    _fields_ = ([(n, _i32) for n in ("act", "E")]
                + [(n, _i64) for n in ("M", "N", "K", "ld_dy", "ld_z", "ld_x", "ld_w", "stride_w", "ld_dx", "ld_dw", "stride_dw")]
                + [(n, _ptr) for n in ("dy", "z", "x", "w", "offsets", "dx", "dw", "db", "workspace")] + [("workspace_bytes", _size)])


_SIGNATURES = {
    "glu_block_norm_fwd": [ctypes.POINTER(NormFwdArgs), _ptr], "glu_block_norm_bwd": [ctypes.POINTER(NormBwdArgs), _ptr],
    "glu_block_norm_bwd_workspace": [_i64, _i64, _i64, ctypes.POINTER(_size)],
    "glu_block_route": [ctypes.POINTER(RouteArgs), _ptr],
    "glu_block_route_workspace": [_i64, _i64, _i32, ctypes.POINTER(_size)],
    "glu_block_dispatch": [ctypes.POINTER(RowsArgs), _ptr], "glu_block_combine": [ctypes.POINTER(RowsArgs), _ptr],
    "glu_block_combine_bwd": [ctypes.POINTER(RowsArgs), _ptr],
    "glu_block_linear_fwd": [ctypes.POINTER(LinearFwdArgs), _ptr], "glu_block_linear_bwd": [ctypes.POINTER(LinearBwdArgs), _ptr],
    "glu_block_linear_fwd_workspace": [ctypes.POINTER(LinearFwdArgs), ctypes.POINTER(_size)],
    "glu_block_linear_bwd_workspace": [ctypes.POINTER(LinearBwdArgs), ctypes.POINTER(_size)],
    "glu_block_device_errors": [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int], "glu_block_abi_version": [],
}
_bound = None
_funcs = {}  # name -> function, filled with the first call


def _c():
    """The library, with this header's signatures set."""
    global _bound
    if _bound is None:
        lib = _lib()
        for name, argtypes in _SIGNATURES.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = argtypes, ctypes.c_int
            _funcs[name] = f
        _bound = lib
    return _bound


def _func(name):
    f = _funcs.get(name)
    if f is None:
        _c()
        f = _funcs[name]
    return f


def _empty_strided(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


# The allocation that torch's own generated code makes (on the current device):
# the same as torch.empty_strided at half its cost per call.
try:
    _alloc = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _alloc = _empty_strided


def _call(name, args, stream):
    st = _func(name)(args, stream)
    if st != GLU_OK:
        raise GluQuantError(st, name)


def _workspace(name, *args):
    n = _size(0)
    st = _func(name)(*args, n)
    if st != GLU_OK:
        raise GluQuantError(st, name)
    return n.value


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()} "
                         "(the kernels run on the current device)")
    return t.device


def _matrix(t, name, shape, device, dtype=_BF16):
    """Checks a matrix and returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    # the stride of a single row is not used, and torch leaves it free
    return st[-2] if shape[-2] > 1 else -(-shape[-1] // 8) * 8


def _rows(t, name, shape, device, dtype=_BF16):
    """A matrix of rows that a call reads, checked, and its row stride: itself, or
    a copy whose rows start on 16 bytes."""
    ld = _matrix(t, name, shape, device, dtype)
    if ld % 8 == 0:
        return t, ld
    t = _new(shape, dtype).copy_(t.detach())
    return t, t.stride(0)


def _packed(t, name, shape, device, dtypes):
    """Checks a contiguous operand."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _new(shape, dtype):
    """A matrix (or a stack of them) whose rows start on 16 bytes, on the
    current device."""
    n = shape[-1]
    ld = n if n % 8 == 0 else -(-n // 8) * 8
    return _alloc(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1), dtype)


def _result(out, key, shape, dtype, device):
    """The matrix for an output: the caller's, checked, or a new one."""
    t = None if out is None else out.get(key)
    if t is None:
        return _new(shape, dtype)
    _matrix(t, key, shape, device, dtype)
    return t


def _result_packed(out, key, shape, dtype, device):
    """The same for a contiguous output."""
    t = None if out is None else out.get(key)
    if t is None:
        return _alloc(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype)
    _packed(t, key, shape, device, (dtype,))
    return t


def _scratch(n):
    return _alloc((n,), (1,), torch.uint8) if n else None


def _ld(t):
    if t is None:
        return 0
    return t.stride(-2) if t.shape[-2] > 1 else -(-t.shape[-1] // 8) * 8


def _p(t):
    return None if t is None else t.data_ptr()


def _on(stream, call, *args, **kwargs):
    """The call with `stream` as torch's current one, so that what it allocates
    belongs to that stream (memory that was freed on another may still be in use
    there)."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _handle(device):
    """The current stream's handle."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _stream_fmt(x, name):
    if x.dtype is _BF16:
        return FMT_BF16
    if x.dtype is _F32:
        return FMT_FP32
    raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")


def _weight_fmt(w_pre, w_post):
    if w_pre is not None and w_post is not None and w_pre.dtype is not w_post.dtype:
        raise TypeError("w_pre and w_post must have the same dtype")
    w = w_pre if w_pre is not None else w_post
    return FMT_FP32 if w is not None and w.dtype is _F32 else FMT_BF16


def _gate(gate, D, device):
    """(rows, row stride) of the gate; a vector counts as one row."""
    if gate is None:
        return 0, 0
    if gate.dim() == 1:
        _packed(gate, "gate", (D,), device, (_BF16,))
        return 1, -(-D // 8) * 8
    return gate.shape[0], _matrix(gate, "gate", (gate.shape[0], D), device)


def block_norm(x, branch=None, *, w_pre=None, w_post=None, gate=None, alpha=1.0, w_offset=0.0, eps=1e-6, out=None, stream=None) -> dict:
    """``r = x + alpha * gate * P(branch)`` and ``y = N(r)``, in one pass.

    ``x`` [M, D] is the residual stream (bf16 or fp32), ``branch`` [M, D] bf16 a
    block's output.  ``w_post`` [D] makes P the RMS norm with weights ``w_post +
    w_offset`` (else P is the branch itself), ``w_pre`` [D] asks for ``y``, the
    RMS norm of r with weights ``w_pre + w_offset`` (both bf16 or both fp32).
    ``gate`` bf16 [D] or [G, D] is shared by M / G consecutive rows each.
    Returns {"r", "y", "rstd_pre", "rstd_post"}, None where not produced: r has
    x's dtype, y is bf16, the rstd [M] fp32 are what ``block_norm_bwd`` wants.
    """
    if stream is not None:
        return _on(stream, block_norm, x, branch, w_pre=w_pre, w_post=w_post, gate=gate, alpha=alpha, w_offset=w_offset, eps=eps, out=out)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    device = _device(x, "x")
    M, D = x.shape
    shape = (M, D)
    fmt = _stream_fmt(x, "x")
    wf = _weight_fmt(w_pre, w_post)
    x, ld_x = _rows(x, "x", shape, device, x.dtype)
    branch, ld_b = _rows(branch, "branch", shape, device) if branch is not None else (None, 0)
    gates, ld_g = _gate(gate, D, device)
    wp = _packed(w_pre, "w_pre", (D,), device, (_BF16, _F32)) if w_pre is not None else None
    wq = _packed(w_post, "w_post", (D,), device, (_BF16, _F32)) if w_post is not None else None
    r = _result(out, "r", shape, x.dtype, device) if branch is not None else None
    y = _result(out, "y", shape, _BF16, device) if wp is not None else None
    rp = _result_packed(out, "rstd_pre", (M,), _F32, device) if wp is not None else None
    rq = _result_packed(out, "rstd_post", (M,), _F32, device) if wq is not None else None
    a = NormFwdArgs(fmt, wf, alpha, w_offset, eps, 0, M, D, gates, ld_x, ld_b, ld_g, _ld(r), _ld(y), x.data_ptr(), _p(branch), _p(gate),
                    wp, wq, _p(r), _p(y), _p(rp), _p(rq))
    _call("glu_block_norm_fwd", a, _handle(device))
    return {"r": r, "y": y, "rstd_pre": rp, "rstd_post": rq}


def block_norm_bwd(r, dy=None, dr=None, *, rstd_pre=None, w_pre=None, branch=None, rstd_post=None, w_post=None, gate=None, alpha=1.0,
                   w_offset=0.0, out=None, stream=None) -> dict:
    """Gradients of ``block_norm``, from those of y (``dy``, given with
    ``w_pre``) and of r (``dr``, or None) and what the forward saved: ``r`` (x
    itself where there was no branch), the rstd and its operands.  Returns
    {"dx", "dw_pre", "dbranch", "dw_post", "dgate"}, None where not produced: dx
    has r's dtype, dbranch is bf16, the gradients of the vectors and of the gate
    ([G, D]) are fp32."""
    if stream is not None:
        return _on(stream, block_norm_bwd, r, dy, dr, rstd_pre=rstd_pre, w_pre=w_pre, branch=branch, rstd_post=rstd_post, w_post=w_post,
                   gate=gate, alpha=alpha, w_offset=w_offset, out=out)
    if r.dim() != 2:
        raise ValueError("r must be a matrix")
    device = _device(r, "r")
    M, D = r.shape
    shape = (M, D)
    fmt = _stream_fmt(r, "r")
    wf = _weight_fmt(w_pre, w_post)
    r, ld_r = _rows(r, "r", shape, device, r.dtype)
    branch, ld_b = _rows(branch, "branch", shape, device) if branch is not None else (None, 0)
    dy, ld_dy = _rows(dy, "dy", shape, device) if dy is not None else (None, 0)
    dr, ld_dr = _rows(dr, "dr", shape, device, r.dtype) if dr is not None else (None, 0)
    gates, ld_g = _gate(gate, D, device)
    wp = _packed(w_pre, "w_pre", (D,), device, (_BF16, _F32)) if w_pre is not None else None
    wq = _packed(w_post, "w_post", (D,), device, (_BF16, _F32)) if w_post is not None else None
    rp = _packed(rstd_pre, "rstd_pre", (M,), device, (_F32,)) if rstd_pre is not None else None
    rq = _packed(rstd_post, "rstd_post", (M,), device, (_F32,)) if rstd_post is not None else None
    dx = _result(out, "dx", shape, r.dtype, device)
    db = _result(out, "dbranch", shape, _BF16, device) if branch is not None else None
    dwp = _result_packed(out, "dw_pre", (D,), _F32, device) if wp is not None else None
    dwq = _result_packed(out, "dw_post", (D,), _F32, device) if wq is not None else None
    dg = _result_packed(out, "dgate", (gates, D), _F32, device) if gates else None
    n = _workspace("glu_block_norm_bwd_workspace", M, D, gates)
    ws = _scratch(n)
    a = NormBwdArgs(fmt, wf, alpha, w_offset, M, D, gates, ld_r, ld_b, ld_g, ld_dy, ld_dr, _ld(dx), _ld(db), r.data_ptr(), _p(branch), _p(gate),
                    wp, wq, rp, rq, _p(dy), _p(dr), dx.data_ptr(), _p(db), _p(dwp), _p(dwq), _p(dg), ws.data_ptr(), n)
    _call("glu_block_norm_bwd", a, _handle(device))
    return {"dx": dx, "dw_pre": dwp, "dbranch": db, "dw_post": dwq, "dgate": dg}


def route(ids, n_experts, *, out=None, stream=None) -> dict:
    """The stable order of the assignments ``ids`` [T, K] (int32 or int64) by
    expert; ids outside [0, n_experts) are dropped.  Returns int32 tensors:
    "slot" [T, K] (the place of each assignment, -1 dropped), "src" [T * K] (the
    assignment t * K + k at each place, -1 past the last) and "offsets"
    [n_experts + 1]."""
    if stream is not None:
        return _on(stream, route, ids, n_experts, out=out)
    device = _device(ids, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, choices]")
    T, K = ids.shape
    shape = (T, K)
    p = _packed(ids, "ids", shape, device, (torch.int64, _I32))
    slot = _result_packed(out, "slot", shape, _I32, device)
    src = _result_packed(out, "src", (T * K,), _I32, device)
    offsets = _result_packed(out, "offsets", (n_experts + 1,), _I32, device)
    n = _workspace("glu_block_route_workspace", T, K, n_experts)
    ws = _scratch(n)
    a = RouteArgs(8 if ids.dtype is torch.int64 else 4, n_experts, T, K, p, slot.data_ptr(), src.data_ptr(), offsets.data_ptr(), _p(ws), n)
    _call("glu_block_route", a, _handle(device))
    return {"slot": slot, "src": src, "offsets": offsets}


def _slots(route, device):
    slot, src = route["slot"], route["src"]
    if slot.dim() != 2:
        raise ValueError("route['slot'] must be [tokens, choices]")
    T, K = slot.shape
    return T, K, _packed(slot, "slot", (T, K), device, (_I32,)), _packed(src, "src", (T * K,), device, (_I32,))


def dispatch(x, route, *, out=None, stream=None):
    """The rows of ``x`` [T, D] in the order of the route, [T * K, D]; rows past
    the last expert's are 0."""
    if stream is not None:
        return _on(stream, dispatch, x, route, out=out)
    device = _device(x, "x")
    T, K, slot, src = _slots(route, device)
    D = x.shape[-1]
    x, ld = _rows(x, "x", (T, D), device)
    xs = _result(None if out is None else {"out": out}, "out", (T * K, D), _BF16, device)
    a = RowsArgs(T, K, D, ld, 0, _ld(xs), 0, slot, src, None, x.data_ptr(), None, None, None, xs.data_ptr(), None)
    _call("glu_block_dispatch", a, _handle(device))
    return xs


def combine(ys, route, weights=None, *, residual=None, out=None, stream=None):
    """``out[t] = residual[t] + sum_k weights[t, k] * ys[slot[t, k]]`` [T, D]
    (``weights`` fp32 [T, K], None: 1; dropped assignments add nothing)."""
    if stream is not None:
        return _on(stream, combine, ys, route, weights, residual=residual, out=out)
    device = _device(ys, "ys")
    T, K, slot, _ = _slots(route, device)
    D = ys.shape[-1]
    ys, ld = _rows(ys, "ys", (T * K, D), device)
    residual, ld_res = _rows(residual, "residual", (T, D), device) if residual is not None else (None, 0)
    w = _packed(weights, "weights", (T, K), device, (_F32,)) if weights is not None else None
    o = _result(None if out is None else {"out": out}, "out", (T, D), _BF16, device)
    a = RowsArgs(T, K, D, _ld(o), ld, 0, ld_res, slot, None, w, None, ys.data_ptr(), _p(residual), o.data_ptr(), None, None)
    _call("glu_block_combine", a, _handle(device))
    return o


def dispatch_bwd(dxs, route, *, out=None, stream=None):
    """Gradient of ``dispatch``: ``dx[t] = sum_k dxs[slot[t, k]]``."""
    return combine(dxs, route, out=out, stream=stream)


def combine_bwd(dout, ys, route, weights, *, out=None, stream=None) -> dict:
    """Gradients of ``combine``: {"dys" [T * K, D] = the weighted rows of
    ``dout`` (0 past the last expert's), "dw" [T, K] fp32 = <ys[slot], dout>};
    the gradient of the residual is ``dout``."""
    if stream is not None:
        return _on(stream, combine_bwd, dout, ys, route, weights, out=out)
    device = _device(dout, "dout")
    T, K, slot, src = _slots(route, device)
    D = dout.shape[-1]
    dout, ld = _rows(dout, "dout", (T, D), device)
    ys, ld_rows = _rows(ys, "ys", (T * K, D), device)
    w = _packed(weights, "weights", (T, K), device, (_F32,))
    dys = _result(out, "dys", (T * K, D), _BF16, device)
    dw = _result_packed(out, "dw", (T, K), _F32, device)
    a = RowsArgs(T, K, D, ld, ld_rows, _ld(dys), 0, slot, src, w, dout.data_ptr(), ys.data_ptr(), None, None, dys.data_ptr(), dw.data_ptr())
    _call("glu_block_combine_bwd", a, _handle(device))
    return {"dys": dys, "dw": dw}


def _weight(w, offsets, K, device):
    """(E, N, row stride, stride between experts, offsets pointer)."""
    if w.dim() == 3:
        E, N = w.shape[0], w.shape[1]
        if offsets is None:
            raise ValueError("weights by expert need the route's offsets")
        ld = _matrix(w, "w", (E, N, K), device)
        return E, N, ld, w.stride(0) if E > 1 else N * ld, _packed(offsets, "offsets", (E + 1,), device, (_I32,))
    if offsets is not None:
        raise ValueError("offsets need weights by expert, [E, N, K]")
    return 0, w.shape[0], _matrix(w, "w", (w.shape[0], K), device), 0, None


def linear(x, w, *, bias=None, act=ACT_IDENTITY, residual=None, offsets=None, keep_z=False, out=None, stream=None) -> dict:
    """``z = x w^T + bias``, ``y = act(z) + residual``: ``x`` [M, K], ``w`` [N, K],
    both bf16.  With ``w`` [E, N, K] and a route's ``offsets`` the rows of expert
    e take ``w[e]`` and ``bias[e]``; rows past the last expert's give 0.  ``bias``
    is bf16 or fp32.  Returns {"y", "z"} (z bf16, None unless ``keep_z``)."""
    if stream is not None:
        return _on(stream, linear, x, w, bias=bias, act=act, residual=residual, offsets=offsets, keep_z=keep_z, out=out)
    device = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    M, K = x.shape
    x, ld_x = _rows(x, "x", (M, K), device)
    E, N, ld_w, stride_w, off = _weight(w, offsets, K, device)
    b = _packed(bias, "bias", (E, N) if E else (N,), device, (_BF16, _F32)) if bias is not None else None
    residual, ld_res = _rows(residual, "residual", (M, N), device) if residual is not None else (None, 0)
    y = _result(out, "y", (M, N), _BF16, device)
    z = _result(out, "z", (M, N), _BF16, device) if keep_z else None
    a = LinearFwdArgs(act, FMT_FP32 if bias is not None and bias.dtype is _F32 else FMT_BF16, E, 0, M, N, K, ld_x, ld_w, stride_w, ld_res,
                      _ld(y), _ld(z), x.data_ptr(), w.data_ptr(), b, _p(residual), off, y.data_ptr(), _p(z), None, 0)
    ws = None
    if E == 0 and M > 16:  # by expert and for few rows it takes none
        n = _workspace("glu_block_linear_fwd_workspace", a)
        if n:
            ws = _scratch(n)
            a.workspace, a.workspace_bytes = ws.data_ptr(), n
    _call("glu_block_linear_fwd", a, _handle(device))
    return {"y": y, "z": z}


def linear_bwd(dy, x, w, *, z=None, act=ACT_IDENTITY, offsets=None, need_dx=True, need_dw=True, need_db=False, out=None, stream=None) -> dict:
    """Gradients of ``linear``: {"dx" bf16 [M, K], "dw" bf16 like ``w``, "db"
    fp32 [N] or [E, N]}, None where not asked for; the gradient of the residual
    is ``dy``.  ``z`` is the forward's where it had an activation."""
    if stream is not None:
        return _on(stream, linear_bwd, dy, x, w, z=z, act=act, offsets=offsets, need_dx=need_dx, need_dw=need_dw, need_db=need_db,
                   out=out)
    device = _device(dy, "dy")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    M, K = x.shape
    x, ld_x = _rows(x, "x", (M, K), device)
    E, N, ld_w, stride_w, off = _weight(w, offsets, K, device)
    dy, ld_dy = _rows(dy, "dy", (M, N), device)
    z, ld_z = _rows(z, "z", (M, N), device) if z is not None else (None, 0)
    dx = _result(out, "dx", (M, K), _BF16, device) if need_dx else None
    dw = _result(out, "dw", tuple(w.shape), _BF16, device) if need_dw else None
    db = _result_packed(out, "db", (E, N) if E else (N,), _F32, device) if need_db else None
    ld_dw = _ld(dw)
    stride_dw = 0 if dw is None or not E else dw.stride(0) if E > 1 else N * ld_dw
    a = LinearBwdArgs(act, E, M, N, K, ld_dy, ld_z, ld_x, ld_w, stride_w, _ld(dx), ld_dw, stride_dw, dy.data_ptr(), _p(z), x.data_ptr(), w.data_ptr(),
                      off, _p(dx), _p(dw), _p(db), None, 0)
    n = _workspace("glu_block_linear_bwd_workspace", a)
    ws = _scratch(n)
    a.workspace, a.workspace_bytes = _p(ws), n
    _call("glu_block_linear_bwd", a, _handle(device))
    return {"dx": dx, "dw": dw, "db": db}


def block_device_errors(clear: bool = False) -> tuple[int, int]:
    """(status, error bits) of the kernels of this module, as ``glu_quant_device_errors``."""
    b = ctypes.c_uint32(0)
    return _c().glu_block_device_errors(ctypes.byref(b), int(clear)), b.value


def block_abi_version() -> int:
    return _c().glu_block_abi_version()
