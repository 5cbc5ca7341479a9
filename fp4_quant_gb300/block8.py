"""A block's products and kept activations in 8-bit floating point with a scale for
each block of 128 (``include/glu_block8.h``), as calls on torch tensors.

An operand is a dict of E4M3 codes (``torch.float8_e4m3fn``) and fp32 scales:

* rows, 1 x 128 blocks: "q" [M, K], "s" [ceil(K / 128), M];
* columns, 128 x 1 blocks, for sums over the rows: "qc" [128 C, K], "sc" [C, K],
  with C = ceil(M / 128) blocks, or M // 128 + E by expert (the rows of expert e
  then begin at block offsets[e] // 128 + e);
* weights, 128 x 128 blocks: "q" [N, K] or [E, N, K], "s" [(E,) ceil(N / 128), ceil(K / 128)].

A block stands for codes times scale; its scale is its largest absolute value (2^-100
at least) over 448, and a NaN or an infinity makes the whole block NaN.  Checks,
allocation, streams and errors are those of ``block``; a matrix of bf16 rows that does
not begin on 16 bytes is copied first as well, such as the second half of a projection
of odd width.  Code matrices have a row stride that is a multiple of 16 and scales are
contiguous.
"""
from __future__ import annotations

import ctypes

import torch

from . import ACT_SILU, FMT_BF16, FMT_FP32, GLU_OK, GluQuantError, _lib
from .block import (_BF16, _F32, _I32, _alloc, _device, _handle, _ld, _matrix, _new, _on, _p, _packed, _result, _rows,
                    _scratch)

__all__ = ["quant8", "quant8_weight", "linear8", "linear8_dx", "linear8_dw", "glu8", "glu8_bwd", "block8_abi_version"]

_F8 = torch.float8_e4m3fn
_i32, _i64, _ptr, _size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


def _fields(dims, pointers, tail):
    return [(n, _i64) for n in dims.split()] + [(n, _ptr) for n in pointers.split()] + tail


class Quant8Args(ctypes.Structure):
    """Mirror of ``glu_block8_quant_args``."""
    _fields_ = _fields("M K ld_x ld_xq ld_q ld_qc", "x xq xs offsets q s qc sc", [("E", _i32), ("reserved", _i32)])


class Quant8WeightArgs(ctypes.Structure):
    """Mirror of ``glu_block8_quant_weight_args``."""
    _fields_ = _fields("N K ld_w stride_w ld_q stride_q", "w q s", [("E", _i32), ("reserved", _i32)])


class Linear8Args(ctypes.Structure):
    """Mirror of ``glu_block8_linear_args``."""
    _fields_ = _fields("M N K ld_x ld_w stride_w ld_y", "xq xs wq ws offsets y workspace",
                       [("workspace_bytes", _size), ("E", _i32), ("grad", _i32)])


class Linear8DwArgs(ctypes.Structure):
    """Mirror of ``glu_block8_linear_dw_args``."""
    _fields_ = _fields("C N K ld_dy ld_x ld_dw stride_dw", "dyq dys xq xs offsets dw workspace",
                       [("workspace_bytes", _size), ("E", _i32), ("dw_fmt", _i32)])


class Glu8Args(ctypes.Structure):
    """Mirror of ``glu_block8_glu_args``."""
    _fields_ = _fields("M H ld_gate ld_up ld_h ld_hq ld_gq ld_uq", "gate up h hq hs gq gs uq us", [("act", _i32), ("reserved", _i32)])


class Glu8BwdArgs(ctypes.Structure):
    """Mirror of ``glu_block8_glu_bwd_args``."""
    _fields_ = _fields("M H ld_gq ld_uq ld_dh ld_d ld_h ld_dq ld_dqc ld_hqc", "gq gs uq us dh offsets d h dq ds dqc dsc hqc hsc",
                       [("act", _i32), ("E", _i32)])


_SIGNATURES = {
    "glu_block8_quant": [ctypes.POINTER(Quant8Args), _ptr], "glu_block8_quant_weight": [ctypes.POINTER(Quant8WeightArgs), _ptr],
    "glu_block8_linear": [ctypes.POINTER(Linear8Args), _ptr], "glu_block8_linear_dw": [ctypes.POINTER(Linear8DwArgs), _ptr],
    "glu_block8_linear_workspace": [ctypes.POINTER(Linear8Args), ctypes.POINTER(_size)],
    "glu_block8_linear_dw_workspace": [ctypes.POINTER(Linear8DwArgs), ctypes.POINTER(_size)],
    "glu_block8_glu": [ctypes.POINTER(Glu8Args), _ptr], "glu_block8_glu_bwd": [ctypes.POINTER(Glu8BwdArgs), _ptr],
    "glu_block8_abi_version": [],
}
_funcs = {}  # name -> function, filled with the first call


def _func(name):
    f = _funcs.get(name)
    if f is None:  # another thread may be half-way through the same
        lib = _lib()
        for n, argtypes in _SIGNATURES.items():
            f = getattr(lib, n)
            f.argtypes, f.restype = argtypes, ctypes.c_int
            _funcs[n] = f
        f = _funcs[name]
    return f


def _call(name, *args):
    st = _func(name)(*args)
    if st != GLU_OK:
        raise GluQuantError(st, name)


def _blocks(n):
    return (n + 127) // 128


def _col_blocks(M, E):
    return M // 128 + E if E else _blocks(M)


def _codes(t, name, shape, device):
    """Checks a code matrix (or a stack) and returns its row stride."""
    _matrix(t, name, shape, device, _F8)
    return t.stride(-2) if shape[-2] > 1 else -(-shape[-1] // 16) * 16


def _scales(t, name, shape, device):
    return _packed(t, name, shape, device, (_F32,))


def _bf16_rows(t, name, shape, device):
    """``_rows``, with a copy too where the base is not on 16 bytes, as the second
    half's of a projection of odd width is not."""
    t, ld = _rows(t, name, shape, device)
    if t.data_ptr() % 16:
        t = _new(shape, _BF16).copy_(t.detach())
        ld = _ld(t)
    return t, ld


def _out_codes(out, key, shape, device):
    """A code matrix for an output (the caller's, checked, or a new one) and its row stride."""
    t = None if out is None else out.get(key)
    if t is None:
        ld = -(-shape[-1] // 16) * 16
        return _alloc(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1), _F8), ld
    return t, _codes(t, key, shape, device)


def _out_scales(out, key, shape, device):
    t = None if out is None else out.get(key)
    if t is None:
        return _alloc(shape, (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1), _F32)
    _scales(t, key, shape, device)
    return t


def _experts(offsets, device):
    """(E, pointer) of a route's offsets, (0, None) without any."""
    if offsets is None:
        return 0, None
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must have one element more than there are experts")
    return offsets.shape[0] - 1, _packed(offsets, "offsets", tuple(offsets.shape), device, (_I32,))


def _row_form(x, name):
    """(M, K, device) of a row form, its codes checked to be on the current device."""
    q = x["q"]
    if q is None or q.dim() != 2:
        raise ValueError(f"{name} must have a row form, {name}['q'] a matrix")
    device = _device(q, f"{name}['q']")
    return q.shape[0], q.shape[1], device


def quant8(x, *, rows=True, cols=False, offsets=None, out=None, stream=None) -> dict:
    """``x`` [M, K] in blocks of 128: its row form ("q", "s"), its column form ("qc",
    "sc"; by expert with a route's ``offsets``), or both from one pass.  ``x`` is a
    bf16 matrix, or a row form (then ``rows=False``): what a forward pass kept,
    cut the other way for the weights' gradient.  Entries not asked for are None."""
    if stream is not None:
        return _on(stream, quant8, x, rows=rows, cols=cols, offsets=offsets, out=out)
    kept = isinstance(x, dict)
    if not rows and not cols:
        raise ValueError("ask for rows, cols or both")
    if kept and rows:
        raise ValueError("x is in row form already (rows=False)")
    if offsets is not None and not cols:
        raise ValueError("offsets cut the column form only")
    if kept:
        M, K, device = _row_form(x, "x")
        xq, xs, ld_xq = x["q"], _scales(x["s"], "x['s']", (_blocks(K), M), device), _codes(x["q"], "x['q']", (M, K), device)
        src, ld = None, 0
    else:
        if x.dim() != 2:
            raise ValueError("x must be a matrix")
        device = _device(x, "x")
        M, K = x.shape
        src, ld = _bf16_rows(x, "x", (M, K), device)
        xq, xs, ld_xq = None, None, 0
    E, off = _experts(offsets, device)
    C = _col_blocks(M, E)
    q, ld_q = _out_codes(out, "q", (M, K), device) if rows else (None, 0)
    s = _out_scales(out, "s", (_blocks(K), M), device) if rows else None
    qc, ld_qc = _out_codes(out, "qc", (128 * C, K), device) if cols else (None, 0)
    sc = _out_scales(out, "sc", (C, K), device) if cols else None
    a = Quant8Args(M, K, ld, ld_xq, ld_q, ld_qc, _p(src), _p(xq), xs, off, _p(q), _p(s), _p(qc), _p(sc), E, 0)
    _call("glu_block8_quant", a, _handle(device))
    return {"q": q, "s": s, "qc": qc, "sc": sc}


def quant8_weight(w, *, out=None, stream=None) -> dict:
    """``w`` bf16 [N, K] or [E, N, K] in blocks of 128 x 128: {"q", "s"}."""
    if stream is not None:
        return _on(stream, quant8_weight, w, out=out)
    if w.dim() not in (2, 3):
        raise ValueError("w must be a matrix or a stack of them")
    device = _device(w, "w")
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 0
    ld_w = _matrix(w, "w", tuple(w.shape), device)
    q, ld_q = _out_codes(out, "q", tuple(w.shape), device)
    s = _out_scales(out, "s", (*w.shape[:-2], _blocks(N), _blocks(K)), device)
    a = Quant8WeightArgs(N, K, ld_w, _stack(w, E, N, ld_w), ld_q, _stack(q, E, N, ld_q), w.data_ptr(), q.data_ptr(), s.data_ptr(), E, 0)
    _call("glu_block8_quant_weight", a, _handle(device))
    return {"q": q, "s": s}


def _stack(t, E, N, ld):
    """Elements between the matrices of a stack."""
    return 0 if not E else t.stride(0) if E > 1 else N * ld


def _may_split(M, E, grad):
    """Whether the library may want a workspace: never by expert, nor for y of one token."""
    return E == 0 and (grad or M > 1)


def _product(x8, w8, offsets, out, grad):
    wq = w8["q"]
    if wq.dim() != (2 if offsets is None else 3):
        raise ValueError("w8['q'] must be [N, K], or [E, N, K] with a route's offsets")
    M, depth, device = _row_form(x8, "x8")
    E, off = _experts(offsets, device)
    N, K = wq.shape[-2:]
    if depth != (N if grad else K):
        raise ValueError(f"x8 has {depth} columns, the weights are {N} x {K}")
    if E and wq.shape[0] != E:
        raise ValueError(f"offsets for {E} experts, weights for {wq.shape[0]}")
    ld_x = _codes(x8["q"], "x8['q']", (M, depth), device)
    xs = _scales(x8["s"], "x8['s']", (_blocks(depth), M), device)
    ld_w = _codes(wq, "w8['q']", tuple(wq.shape), device)
    ws = _scales(w8["s"], "w8['s']", (*wq.shape[:-2], _blocks(N), _blocks(K)), device)
    y = _result(None if out is None else {"out": out}, "out", (M, K if grad else N), _BF16, device)
    a = Linear8Args(M, N, K, ld_x, ld_w, _stack(wq, E, N, ld_w), _ld(y), x8["q"].data_ptr(), xs, wq.data_ptr(), ws, off, y.data_ptr(),
                    None, 0, E, int(grad))
    ws = None
    if _may_split(M, E, grad):
        n = _size(0)
        _call("glu_block8_linear_workspace", a, n)
        ws = _scratch(n.value)
        a.workspace, a.workspace_bytes = _p(ws), n.value
    _call("glu_block8_linear", a, _handle(device))
    return y


def linear8(x8, w8, *, offsets=None, out=None, stream=None):
    """``x w^T`` bf16 [M, N] of ``x8`` [M, K] (row form) and ``w8`` [N, K] (weights);
    with ``w8`` [E, N, K] and a route's ``offsets`` the rows of expert e take
    ``w[e]``, rows past the last expert's give 0."""
    if stream is not None:
        return _on(stream, linear8, x8, w8, offsets=offsets, out=out)
    return _product(x8, w8, offsets, out, False)


def linear8_dx(dy8, w8, *, offsets=None, out=None, stream=None):
    """Gradient of ``linear8``'s x: ``dy w`` bf16 [M, K] of ``dy8`` [M, N] (row form)
    and the same ``w8``."""
    if stream is not None:
        return _on(stream, linear8_dx, dy8, w8, offsets=offsets, out=out)
    return _product(dy8, w8, offsets, out, True)


def linear8_dw(dy8, x8, *, offsets=None, dtype=torch.bfloat16, out=None, stream=None):
    """Gradient of ``linear8``'s w: ``dy^T x`` [N, K], or by expert [E, N, K], in
    ``dtype`` (bf16 or fp32), of the column forms of dy and x (with the same
    ``offsets``).  Experts without rows get 0."""
    if stream is not None:
        return _on(stream, linear8_dw, dy8, x8, offsets=offsets, dtype=dtype, out=out)
    dyq, xq = dy8["qc"], x8["qc"]
    if dyq is None or xq is None or dyq.dim() != 2 or xq.dim() != 2 or dyq.shape[0] != xq.shape[0] or dyq.shape[0] % 128:
        raise ValueError("dy8 and x8 must have column forms: dy8['qc'] and x8['qc'] of the same number of rows, a multiple of 128")
    if dtype not in (_BF16, _F32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    device = _device(dyq, "dy8['qc']")
    E, off = _experts(offsets, device)
    C, N, K = dyq.shape[0] // 128, dyq.shape[1], xq.shape[1]
    ld_dy, ld_x = _codes(dyq, "dy8['qc']", (128 * C, N), device), _codes(xq, "x8['qc']", (128 * C, K), device)
    dys, xs = _scales(dy8["sc"], "dy8['sc']", (C, N), device), _scales(x8["sc"], "x8['sc']", (C, K), device)
    dw = _result(None if out is None else {"out": out}, "out", (E, N, K) if E else (N, K), dtype, device)
    ld = _ld(dw)
    a = Linear8DwArgs(C, N, K, ld_dy, ld_x, ld, _stack(dw, E, N, ld), dyq.data_ptr(), dys, xq.data_ptr(), xs, off, dw.data_ptr(), None, 0,
                      E, FMT_FP32 if dtype is _F32 else FMT_BF16)
    n = _size(0)
    _call("glu_block8_linear_dw_workspace", a, n)
    ws = _scratch(n.value)
    a.workspace, a.workspace_bytes = _p(ws), n.value
    _call("glu_block8_linear_dw", a, _handle(device))
    return dw


def _some(out, key):
    return None if out is None else out.get(key)


def glu8(gate, up, *, act=ACT_SILU, h8=True, out=None, stream=None) -> dict:
    """``h = act(gate) * up`` of bf16 [M, H] matrices, with gate and up kept in 8
    bits: {"h", "gate", "up"}, the latter two in row form, h in row form
    (quantised from its unrounded values) or, with ``h8=False``, as bf16."""
    if stream is not None:
        return _on(stream, glu8, gate, up, act=act, h8=h8, out=out)
    if gate.dim() != 2:
        raise ValueError("gate must be a matrix")
    device = _device(gate, "gate")
    M, H = gate.shape
    gate, ld_gate = _bf16_rows(gate, "gate", (M, H), device)
    up, ld_up = _bf16_rows(up, "up", (M, H), device)
    got, lds = {}, {}
    for key in ("h", "gate", "up") if h8 else ("gate", "up"):
        q, lds[key] = _out_codes(_some(out, key), "q", (M, H), device)
        got[key] = {"q": q, "s": _out_scales(_some(out, key), "s", (_blocks(H), M), device)}
    g, u = got["gate"], got["up"]
    if h8:
        h = None
        hq, hs = _p(got["h"]["q"]), _p(got["h"]["s"])
    else:
        h, hq, hs = _result(out, "h", (M, H), _BF16, device), None, None
        got = {"h": h, **got}
    a = Glu8Args(M, H, ld_gate, ld_up, _ld(h), lds.get("h", 0), lds["gate"], lds["up"], gate.data_ptr(), up.data_ptr(), _p(h), hq, hs,
                 g["q"].data_ptr(), g["s"].data_ptr(), u["q"].data_ptr(), u["s"].data_ptr(), act, 0)
    _call("glu_block8_glu", a, _handle(device))
    return got


def glu8_bwd(gate8, up8, dh, *, act=ACT_SILU, quant=False, need_h=True, offsets=None, out=None, stream=None) -> dict:
    """Backward of ``glu8`` from what it kept and ``dh`` bf16 [M, H]: {"d", "h"} with
    ``d = [dh * up * act'(gate) | dh * act(gate)]`` [M, 2 H] and ``h = act(gate) * up``
    (None unless ``need_h``), gate and up being what the 8 bits stand for.

    As bf16, or with ``quant`` as the operands of the products that follow: d in
    row and column form ({"q", "s", "qc", "sc"}), h in column form, the column
    forms by expert with a route's ``offsets``; H is then a multiple of 128."""
    if stream is not None:
        return _on(stream, glu8_bwd, gate8, up8, dh, act=act, quant=quant, need_h=need_h, offsets=offsets, out=out)
    M, H, device = _row_form(gate8, "gate8")
    ld_gq, ld_uq = _codes(gate8["q"], "gate8['q']", (M, H), device), _codes(up8["q"], "up8['q']", (M, H), device)
    gs, us = _scales(gate8["s"], "gate8['s']", (_blocks(H), M), device), _scales(up8["s"], "up8['s']", (_blocks(H), M), device)
    dh, ld_dh = _bf16_rows(dh, "dh", (M, H), device)
    if offsets is not None and not quant:
        raise ValueError("offsets cut the column forms of quant=True only")
    E, off = _experts(offsets, device)
    a = Glu8BwdArgs(M, H, ld_gq, ld_uq, ld_dh, 0, 0, 0, 0, 0, gate8["q"].data_ptr(), gs, up8["q"].data_ptr(), us, dh.data_ptr(), off)
    a.act, a.E = act, E
    if quant:
        C = _col_blocks(M, E)
        od, oh = _some(out, "d"), _some(out, "h")
        q, a.ld_dq = _out_codes(od, "q", (M, 2 * H), device)
        s = _out_scales(od, "s", (_blocks(2 * H), M), device)
        qc, a.ld_dqc = _out_codes(od, "qc", (128 * C, 2 * H), device)
        sc = _out_scales(od, "sc", (C, 2 * H), device)
        d, h = {"q": q, "s": s, "qc": qc, "sc": sc}, None
        a.dq, a.ds, a.dqc, a.dsc = q.data_ptr(), s.data_ptr(), qc.data_ptr(), sc.data_ptr()
        if need_h:
            hqc, a.ld_hqc = _out_codes(oh, "qc", (128 * C, H), device)
            h = {"qc": hqc, "sc": _out_scales(oh, "sc", (C, H), device)}
            a.hqc, a.hsc = hqc.data_ptr(), h["sc"].data_ptr()
    else:
        d = _result(out, "d", (M, 2 * H), _BF16, device)
        h = _result(out, "h", (M, H), _BF16, device) if need_h else None
        a.d, a.h, a.ld_d, a.ld_h = d.data_ptr(), _p(h), _ld(d), _ld(h)
    _call("glu_block8_glu_bwd", a, _handle(device))
    return {"d": d, "h": h}


def block8_abi_version() -> int:
    return _func("glu_block8_abi_version")()
