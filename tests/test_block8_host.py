"""Host-side checks of the 8-bit operators' C ABI and binding (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import fp4_quant_gb300 as G
from fp4_quant_gb300 import block8 as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "glu_block8.h")
P = 1 << 12  # a 16-byte aligned placeholder address (never dereferenced)
STRUCTS = {"glu_block8_quant_args": B.Quant8Args, "glu_block8_quant_weight_args": B.Quant8WeightArgs, "glu_block8_linear_args": B.Linear8Args,
           "glu_block8_linear_dw_args": B.Linear8DwArgs, "glu_block8_glu_args": B.Glu8Args, "glu_block8_glu_bwd_args": B.Glu8BwdArgs}


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"GLU_API\s+int\s+(glu_block8_\w+)\s*\(", open(HEADER).read()))
    assert names == set(B._SIGNATURES)
    lib = ctypes.CDLL(G.library_path())
    assert all(hasattr(lib, n) for n in names)
    assert G.block8_abi_version() == 1


def test_binding_mirrors_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "glu_block8.h"', "int main(void) {"]
    for st, cls in STRUCTS.items():
        lines.append(f'  printf("{st} %zu\\n", sizeof({st}));')
        lines += [f'  printf("{st}.{n} %zu\\n", offsetof({st}, {n}));' for n, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.splitlines())
    for st, cls in STRUCTS.items():
        assert int(got[st]) == ctypes.sizeof(cls), st
        for n, _ in cls._fields_:
            assert int(got[f"{st}.{n}"]) == getattr(cls, n).offset, (st, n)


def _status(name, cls, base, kw):
    return B._func(name)(ctypes.byref(cls(**{**base, **kw})), None)


QUANT = dict(M=300, K=64, ld_x=64, ld_xq=64, ld_q=64, ld_qc=64, x=P, q=P, s=P, qc=P, sc=P)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), G.GLU_EINVAL), (dict(K=0), G.GLU_EINVAL), (dict(x=None), G.GLU_EINVAL), (dict(xq=P, xs=P), G.GLU_EINVAL),
    (dict(x=None, xq=P, xs=P), G.GLU_EINVAL), (dict(x=None, xq=P, q=None, s=None), G.GLU_EINVAL), (dict(s=None), G.GLU_EINVAL),
    (dict(sc=None), G.GLU_EINVAL), (dict(q=None, s=None, qc=None, sc=None), G.GLU_EINVAL), (dict(reserved=1), G.GLU_EINVAL),
    (dict(E=-1), G.GLU_EINVAL), (dict(E=4), G.GLU_EINVAL), (dict(offsets=P), G.GLU_EINVAL), (dict(E=4, offsets=P, qc=None, sc=None), G.GLU_EINVAL),
    (dict(E=1025, offsets=P), G.GLU_ESHAPE), (dict(M=1 << 31), G.GLU_ESHAPE), (dict(K=(1 << 23) + 1), G.GLU_ESHAPE), (dict(ld_q=32), G.GLU_ESHAPE),
    (dict(M=(1 << 31) - 1025, K=1 << 23, ld_x=1 << 23, ld_q=1 << 23, ld_qc=1 << 23), G.GLU_ESHAPE),
    (dict(ld_qc=72), G.GLU_EALIGN), (dict(ld_x=68), G.GLU_EALIGN), (dict(x=P + 8), G.GLU_EALIGN), (dict(sc=P + 2), G.GLU_EALIGN)])
def test_quant_refusals(kw, status):
    assert _status("glu_block8_quant", B.Quant8Args, QUANT, kw) == status


WEIGHT = dict(N=64, K=64, ld_w=64, stride_w=4096, ld_q=64, stride_q=4096, w=P, q=P, s=P, E=2)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), G.GLU_EINVAL), (dict(w=None), G.GLU_EINVAL), (dict(s=None), G.GLU_EINVAL), (dict(E=-1), G.GLU_EINVAL), (dict(reserved=2), G.GLU_EINVAL),
    (dict(E=1025), G.GLU_ESHAPE), (dict(stride_w=4088), G.GLU_ESHAPE), (dict(ld_q=48), G.GLU_ESHAPE),
    (dict(N=1 << 23, K=1 << 23, ld_w=1 << 23, ld_q=1 << 23, E=0), G.GLU_ESHAPE),
    (dict(stride_q=4104), G.GLU_EALIGN), (dict(ld_w=70, stride_w=8192), G.GLU_EALIGN), (dict(q=P + 8), G.GLU_EALIGN)])
def test_quant_weight_refusals(kw, status):
    assert _status("glu_block8_quant_weight", B.Quant8WeightArgs, WEIGHT, kw) == status


LINEAR = dict(M=64, N=32, K=64, ld_x=64, ld_w=64, stride_w=2048 + 64, ld_y=64, xq=P, xs=P, wq=P, ws=P, y=P, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), G.GLU_EINVAL), (dict(grad=2), G.GLU_EINVAL), (dict(xs=None), G.GLU_EINVAL), (dict(ws=None), G.GLU_EINVAL), (dict(y=None), G.GLU_EINVAL),
    (dict(E=2), G.GLU_EINVAL), (dict(offsets=P), G.GLU_EINVAL), (dict(M=1 << 31), G.GLU_ESHAPE), (dict(N=(1 << 23) + 1), G.GLU_ESHAPE),
    (dict(ld_x=48), G.GLU_ESHAPE), (dict(grad=1, ld_y=56), G.GLU_ESHAPE), (dict(E=2, offsets=P, stride_w=1024), G.GLU_ESHAPE),
    (dict(ld_w=72), G.GLU_EALIGN), (dict(ld_y=68), G.GLU_EALIGN), (dict(xq=P + 8), G.GLU_EALIGN), (dict(ws=P + 2), G.GLU_EALIGN),
    (dict(E=2, offsets=P, stride_w=2056), G.GLU_EALIGN)])
def test_linear_refusals(kw, status):
    assert _status("glu_block8_linear", B.Linear8Args, LINEAR, kw) == status


def test_linear_workspace():
    """Parts of split sums: none for few tokens, by expert and where tiles abound."""
    def need(**kw):
        n = ctypes.c_size_t(99)
        assert B._func("glu_block8_linear_workspace")(ctypes.byref(B.Linear8Args(**{**LINEAR, **kw})), ctypes.byref(n)) == G.GLU_OK
        return n.value
    big = dict(N=1030, K=8192, ld_x=8192, ld_w=8192, ld_y=1032)
    assert need(M=16, **big) == 0 and need(M=4096, **big) == 0 and need(M=200, E=4, **big) == 0
    n = need(M=200, **big)
    assert n > 0 and n % (200 * 1032 * 4) == 0
    assert need(M=200, N=8192, K=1030, grad=1) == n
    assert _status("glu_block8_linear", B.Linear8Args, LINEAR, dict(M=200, **big, workspace_bytes=n - 1)) == G.GLU_EINVAL
    assert _status("glu_block8_linear", B.Linear8Args, LINEAR, dict(M=200, **big, workspace=None)) == G.GLU_EINVAL
    assert _status("glu_block8_linear", B.Linear8Args, LINEAR, dict(M=200, **big, workspace=P + 8, workspace_bytes=n)) == G.GLU_EALIGN


DW = dict(C=3, N=32, K=64, ld_dy=32, ld_x=64, ld_dw=64, stride_dw=2048, dyq=P, dys=P, xq=P, xs=P, dw=P, dw_fmt=2, workspace=P, workspace_bytes=1 << 40)


def test_linear_dw_workspace():
    """Parts of split sums where the tiles are few and the sum is long."""
    def need(**kw):
        n = ctypes.c_size_t(99)
        assert B._func("glu_block8_linear_dw_workspace")(ctypes.byref(B.Linear8DwArgs(**{**DW, **kw})), ctypes.byref(n)) == G.GLU_OK
        return n.value
    few = dict(C=32, N=1024, K=1023, ld_dy=1024, ld_x=1024, ld_dw=1024)
    n = need(**few)
    assert n > 0 and n % (1024 * 1024 * 4) == 0 and need(**{**few, "dw_fmt": 3}) == n
    assert need(**{**few, "C": 3}) == 0 and need(C=32, N=8192, K=8192) == 0 and need(C=300, N=2048, K=2048, E=64) == 0
    assert need(C=260, N=300, K=300, E=4) % (4 * 300 * 304 * 4) == 0 and need(C=260, N=300, K=300, E=4) > 0
    for kw, status in [(dict(workspace=None), G.GLU_EINVAL), (dict(workspace_bytes=n - 1), G.GLU_EINVAL), (dict(workspace=P + 8), G.GLU_EALIGN)]:
        assert _status("glu_block8_linear_dw", B.Linear8DwArgs, DW, {**few, **kw}) == status


@pytest.mark.parametrize("kw,status", [
    (dict(C=0), G.GLU_EINVAL), (dict(dw_fmt=0), G.GLU_EINVAL), (dict(dys=None), G.GLU_EINVAL), (dict(dw=None), G.GLU_EINVAL),
    (dict(E=2), G.GLU_EINVAL), (dict(E=4, offsets=P), G.GLU_EINVAL), (dict(C=1 << 24), G.GLU_ESHAPE), (dict(ld_dw=56), G.GLU_ESHAPE),
    (dict(E=2, offsets=P, stride_dw=1024), G.GLU_ESHAPE), (dict(ld_dy=56), G.GLU_EALIGN), (dict(ld_dw=68), G.GLU_EALIGN), (dict(xs=P + 2), G.GLU_EALIGN)])
def test_linear_dw_refusals(kw, status):
    assert _status("glu_block8_linear_dw", B.Linear8DwArgs, DW, kw) == status


GLU = dict(M=64, H=48, ld_gate=48, ld_up=48, ld_h=48, ld_hq=48, ld_gq=48, ld_uq=48, gate=P, up=P, hq=P, hs=P, gq=P, gs=P, uq=P, us=P)


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), G.GLU_EINVAL), (dict(act=16), G.GLU_EINVAL), (dict(M=0), G.GLU_EINVAL), (dict(gate=None), G.GLU_EINVAL), (dict(us=None), G.GLU_EINVAL),
    (dict(h=P), G.GLU_EINVAL), (dict(hq=None), G.GLU_EINVAL), (dict(hs=None), G.GLU_EINVAL), (dict(reserved=1), G.GLU_EINVAL),
    (dict(H=(1 << 23) + 1), G.GLU_ESHAPE), (dict(ld_up=40), G.GLU_ESHAPE), (dict(ld_gq=56), G.GLU_EALIGN), (dict(ld_gate=52), G.GLU_EALIGN),
    (dict(gs=P + 2), G.GLU_EALIGN)])
def test_glu_refusals(kw, status):
    assert _status("glu_block8_glu", B.Glu8Args, GLU, kw) == status


GLU_BWD = dict(M=64, H=128, ld_gq=128, ld_uq=128, ld_dh=128, ld_d=256, ld_h=128, ld_dq=256, ld_dqc=256, ld_hqc=128, gq=P, gs=P, uq=P, us=P, dh=P)
PLAIN, QUANTISED = dict(d=P, h=P), dict(dq=P, ds=P, dqc=P, dsc=P, hqc=P, hsc=P)


@pytest.mark.parametrize("kw,status", [
    (dict(**PLAIN, act=5), G.GLU_EINVAL), (dict(**PLAIN, dh=None), G.GLU_EINVAL), (dict(**PLAIN, **QUANTISED), G.GLU_EINVAL), (dict(), G.GLU_EINVAL),
    (dict(**PLAIN, E=1, offsets=P), G.GLU_EINVAL), (dict(**{**QUANTISED, "ds": None}), G.GLU_EINVAL), (dict(**{**QUANTISED, "hsc": None}), G.GLU_EINVAL),
    (dict(**QUANTISED, h=P), G.GLU_EINVAL), (dict(**QUANTISED, E=3), G.GLU_EINVAL), (dict(**QUANTISED, H=64), G.GLU_ESHAPE),
    (dict(**PLAIN, H=(1 << 22) + 128), G.GLU_ESHAPE), (dict(**PLAIN, ld_d=248), G.GLU_ESHAPE), (dict(**QUANTISED, ld_hqc=112), G.GLU_ESHAPE),
    (dict(**QUANTISED, ld_dq=264), G.GLU_EALIGN), (dict(**PLAIN, ld_dh=132), G.GLU_EALIGN), (dict(**{**QUANTISED, "dsc": P + 2}), G.GLU_EALIGN)])
def test_glu_bwd_refusals(kw, status):
    assert _status("glu_block8_glu_bwd", B.Glu8BwdArgs, GLU_BWD, kw) == status


def test_null_arguments():
    for name in B._SIGNATURES:
        if name.endswith("_workspace"):
            a = B.Linear8DwArgs(**DW) if "dw" in name else B.Linear8Args(**LINEAR)
            assert B._func(name)(ctypes.byref(a), None) == G.GLU_EINVAL
        elif name != "glu_block8_abi_version":
            assert B._func(name)(None, None) == G.GLU_EINVAL


def test_accepted_arguments_get_as_far_as_the_device():
    if torch.cuda.is_available():
        pytest.skip("placeholder addresses must not reach a device")
    for name, cls, base in [("glu_block8_quant", B.Quant8Args, QUANT), ("glu_block8_quant", B.Quant8Args, {**QUANT, "E": 300, "offsets": P}),
                            ("glu_block8_quant_weight", B.Quant8WeightArgs, WEIGHT),
                            ("glu_block8_linear", B.Linear8Args, LINEAR), ("glu_block8_linear", B.Linear8Args, {**LINEAR, "grad": 1}),
                            ("glu_block8_linear_dw", B.Linear8DwArgs, DW), ("glu_block8_linear_dw", B.Linear8DwArgs, {**DW, "dw_fmt": 3}),
                            ("glu_block8_glu", B.Glu8Args, GLU), ("glu_block8_glu_bwd", B.Glu8BwdArgs, {**GLU_BWD, **PLAIN}),
                            ("glu_block8_glu_bwd", B.Glu8BwdArgs, {**GLU_BWD, **QUANTISED})]:
        assert _status(name, cls, base, {}) == G.GLU_EDEVICE


def test_binding_refuses_on_the_cpu():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    row = {"q": torch.zeros(4, 16, dtype=torch.float8_e4m3fn), "s": torch.ones(1, 4)}
    for call in (lambda: G.quant8(x), lambda: G.quant8_weight(x), lambda: G.linear8(row, row), lambda: G.linear8_dx(row, row),
                 lambda: G.linear8_dw({"qc": torch.zeros(128, 16, dtype=torch.float8_e4m3fn)}, {"qc": torch.zeros(128, 16, dtype=torch.float8_e4m3fn)}),
                 lambda: G.glu8(x, x), lambda: G.glu8_bwd(row, row, x), lambda: G.quant8(row, rows=False, cols=True)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="rows=False"):
        G.quant8(row)
    with pytest.raises(ValueError, match="rows, cols"):
        G.quant8(x, rows=False)
    with pytest.raises(ValueError, match="column form"):
        G.quant8(x, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="offsets"):
        G.linear8(row, {"q": torch.zeros(2, 4, 16, dtype=torch.float8_e4m3fn), "s": torch.ones(2, 1, 1)})
    with pytest.raises(TypeError, match="dtype"):
        G.linear8_dw({"qc": torch.zeros(128, 16)}, {"qc": torch.zeros(128, 16)}, dtype=torch.float16)
    with pytest.raises(ValueError, match="row form"):
        G.linear8({"q": None, "s": None}, row)
    with pytest.raises(ValueError, match="column forms"):
        G.linear8_dw({"qc": None, "sc": None}, {"qc": None, "sc": None})
    with pytest.raises(ValueError, match="128"):
        G.linear8_dw({"qc": torch.zeros(100, 16)}, {"qc": torch.zeros(100, 16)})


@pytest.mark.parametrize("N,K", [(512, 300), (2048, 2048), (300, 8192), (8192, 7168)])
def test_binding_asks_for_every_workspace(N, K):
    """A call for which the library wants a workspace is one for which the binding asks."""
    seen = set()
    for grad in (False, True):
        for E in (0, 3):
            for M in (*range(1, 21), 200, 4096):
                n = ctypes.c_size_t(0)
                a = B.Linear8Args(M=M, N=N, K=K, E=E, grad=int(grad))
                assert B._func("glu_block8_linear_workspace")(ctypes.byref(a), ctypes.byref(n)) == G.GLU_OK
                assert n.value == 0 or B._may_split(M, E, grad), (M, E, grad, n.value)
                seen.add((M == 1, grad, n.value > 0))
    if N >= 2048:
        assert (True, True, True) in seen  # a gradient of one token does take one


def test_first_calls_from_several_threads(monkeypatch):
    """A thread may find the table of functions half filled by another one: it fills the rest."""
    first = next(iter(B._SIGNATURES))
    monkeypatch.setattr(B, "_funcs", {first: B._func(first)})
    for name, argtypes in B._SIGNATURES.items():
        assert B._func(name).argtypes == argtypes
    assert B._func("glu_block8_abi_version")() == 1
