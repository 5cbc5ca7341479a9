"""Host-side checks of the block operators' C ABI and binding (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

import fp4_quant_gb300 as G
from fp4_quant_gb300 import block as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "glu_block.h")
P = 1 << 12  # a 16-byte aligned placeholder address (never dereferenced)
STRUCTS = {"glu_block_norm_fwd_args": B.NormFwdArgs, "glu_block_norm_bwd_args": B.NormBwdArgs, "glu_block_route_args": B.RouteArgs,
           "glu_block_rows_args": B.RowsArgs, "glu_block_linear_fwd_args": B.LinearFwdArgs, "glu_block_linear_bwd_args": B.LinearBwdArgs}


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"GLU_API\s+int\s+(glu_block_\w+)\s*\(", open(HEADER).read()))
    assert names == set(B._SIGNATURES)
    lib = ctypes.CDLL(G.library_path())
    assert all(hasattr(lib, n) for n in names)
    assert G.block_abi_version() == 1


def test_binding_mirrors_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "glu_block.h"', "int main(void) {"]
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
    return getattr(B._c(), name)(ctypes.byref(cls(**{**base, **kw})), None)


NORM = dict(x_fmt=2, w_fmt=2, alpha=1.0, w_offset=0.0, eps=1e-6, reserved=0, M=8, D=64, gates=2, ld_x=64, ld_branch=64, ld_gate=64, ld_r=64,
            ld_y=64, x=P, branch=P, gate=P, w_pre=P, w_post=P, r=P, y=P, rstd_pre=P, rstd_post=P)


@pytest.mark.parametrize("kw,status", [
    (dict(x_fmt=0), G.GLU_EINVAL), (dict(w_fmt=1), G.GLU_EINVAL), (dict(reserved=1), G.GLU_EINVAL), (dict(M=0), G.GLU_EINVAL),
    (dict(x=None), G.GLU_EINVAL), (dict(branch=None), G.GLU_EINVAL), (dict(r=None), G.GLU_EINVAL), (dict(y=None), G.GLU_EINVAL),
    (dict(rstd_post=None), G.GLU_EINVAL), (dict(gate=None), G.GLU_EINVAL), (dict(gates=0), G.GLU_EINVAL), (dict(w_pre=None), G.GLU_EINVAL),
    (dict(gates=3), G.GLU_ESHAPE), (dict(ld_x=56), G.GLU_ESHAPE), (dict(M=1 << 60), G.GLU_ESHAPE),
    (dict(D=32776, ld_x=32776, ld_branch=32776, ld_gate=32776, ld_r=32776, ld_y=32776), G.GLU_ESHAPE),
    (dict(ld_y=68), G.GLU_EALIGN), (dict(x=P + 8), G.GLU_EALIGN), (dict(w_pre=P + 4), G.GLU_EALIGN)])
def test_norm_fwd_refusals(kw, status):
    assert _status("glu_block_norm_fwd", B.NormFwdArgs, NORM, kw) == status


NORM_BWD = dict(x_fmt=2, w_fmt=2, alpha=1.0, w_offset=0.0, M=8, D=64, gates=2, ld_r=64, ld_branch=64, ld_gate=64, ld_dy=64, ld_dr=64, ld_dx=64,
                ld_dbranch=64, r=P, branch=P, gate=P, w_pre=P, w_post=P, rstd_pre=P, rstd_post=P, dy=P, dr=P, dx=P, dbranch=P, dw_pre=P,
                dw_post=P, dgate=P, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(dx=None), G.GLU_EINVAL), (dict(dy=None), G.GLU_EINVAL), (dict(rstd_pre=None), G.GLU_EINVAL), (dict(dgate=None), G.GLU_EINVAL),
    (dict(dbranch=None), G.GLU_EINVAL), (dict(workspace=None), G.GLU_EINVAL), (dict(workspace_bytes=16), G.GLU_EINVAL),
    (dict(w_pre=None, dy=None, dw_pre=None, dr=None), G.GLU_EINVAL), (dict(gates=5), G.GLU_ESHAPE), (dict(ld_dr=8), G.GLU_ESHAPE),
    (dict(D=16392), G.GLU_ESHAPE), (dict(ld_dx=65), G.GLU_EALIGN), (dict(dgate=P + 4), G.GLU_EALIGN)])
def test_norm_bwd_refusals(kw, status):
    assert _status("glu_block_norm_bwd", B.NormBwdArgs, NORM_BWD, kw) == status


ROUTE = dict(id_bytes=8, E=8, T=16, K=2, ids=P, slot=P, src=P, offsets=P, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(id_bytes=2), G.GLU_EINVAL), (dict(T=0), G.GLU_EINVAL), (dict(E=0), G.GLU_EINVAL), (dict(ids=None), G.GLU_EINVAL),
    (dict(T=4096, workspace_bytes=0), G.GLU_EINVAL), (dict(E=1025), G.GLU_ESHAPE), (dict(T=1 << 31), G.GLU_ESHAPE), (dict(slot=P + 4), G.GLU_EALIGN)])
def test_route_refusals(kw, status):
    assert _status("glu_block_route", B.RouteArgs, ROUTE, kw) == status


ROWS = dict(T=16, K=2, D=64, ld_tokens=64, ld_rows=64, ld_rows_out=64, ld_residual=64, slot=P)


@pytest.mark.parametrize("name,base,kw,status", [
    ("dispatch", dict(src=P, tokens_in=P, rows_out=P), dict(rows_in=P), G.GLU_EINVAL),
    ("dispatch", dict(src=P, tokens_in=P, rows_out=P), dict(w=P), G.GLU_EINVAL),
    ("dispatch", dict(src=P, tokens_in=P, rows_out=P), dict(src=None), G.GLU_EINVAL),
    ("dispatch", dict(src=P, tokens_in=P, rows_out=P), dict(ld_rows_out=56), G.GLU_ESHAPE),
    ("dispatch", dict(src=P, tokens_in=P, rows_out=P), dict(ld_tokens=70), G.GLU_EALIGN),
    ("combine", dict(rows_in=P, tokens_out=P), dict(tokens_out=None), G.GLU_EINVAL),
    ("combine", dict(rows_in=P, tokens_out=P), dict(K=1 << 31), G.GLU_ESHAPE),
    ("combine", dict(rows_in=P, tokens_out=P), dict(residual=P + 2), G.GLU_EALIGN),
    ("combine_bwd", dict(src=P, w=P, tokens_in=P, rows_in=P, rows_out=P, dw=P), dict(w=None), G.GLU_EINVAL),
    ("combine_bwd", dict(src=P, w=P, tokens_in=P, rows_in=P, rows_out=P, dw=P), dict(residual=P), G.GLU_EINVAL),
    ("combine_bwd", dict(src=P, w=P, tokens_in=P, rows_in=P, rows_out=P, dw=P), dict(dw=P + 4), G.GLU_EALIGN)])
def test_rows_refusals(name, base, kw, status):
    assert _status("glu_block_" + name, B.RowsArgs, {**ROWS, **base}, kw) == status


LIN = dict(act=3, b_fmt=2, E=0, M=16, N=64, K=64, ld_x=64, ld_w=64, stride_w=0, ld_residual=64, ld_y=64, ld_z=64, x=P, w=P, y=P,
           workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), G.GLU_EINVAL), (dict(act=16), G.GLU_EINVAL), (dict(b_fmt=0), G.GLU_EINVAL), (dict(M=0), G.GLU_EINVAL), (dict(w=None), G.GLU_EINVAL),
    (dict(offsets=P), G.GLU_EINVAL), (dict(E=4, stride_w=4096), G.GLU_EINVAL), (dict(E=1025), G.GLU_ESHAPE), (dict(ld_w=56), G.GLU_ESHAPE),
    (dict(E=4, offsets=P, stride_w=64), G.GLU_ESHAPE), (dict(M=1 << 31), G.GLU_ESHAPE), (dict(M=1 << 28, N=1 << 20, ld_y=1 << 20), G.GLU_ESHAPE),
    (dict(E=4, offsets=P, stride_w=4100), G.GLU_EALIGN), (dict(ld_x=68), G.GLU_EALIGN), (dict(bias=P + 2), G.GLU_EALIGN)])
def test_linear_fwd_refusals(kw, status):
    assert _status("glu_block_linear_fwd", B.LinearFwdArgs, LIN, kw) == status


LIN_BWD = dict(act=3, E=0, M=16, N=64, K=64, ld_dy=64, ld_z=64, ld_x=64, ld_w=64, stride_w=0, ld_dx=64, ld_dw=64, stride_dw=0, dy=P, x=P, w=P, dx=P,
               dw=P, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(z=P), G.GLU_EINVAL), (dict(act=0), G.GLU_EINVAL), (dict(dx=None, dw=None), G.GLU_EINVAL), (dict(w=None), G.GLU_EINVAL),
    (dict(x=None), G.GLU_EINVAL), (dict(act=0, z=P, workspace_bytes=8), G.GLU_EINVAL), (dict(db=P, workspace=None), G.GLU_EINVAL),
    (dict(E=2, offsets=P, stride_w=4096, stride_dw=100), G.GLU_ESHAPE), (dict(ld_dw=72, dw=P + 8), G.GLU_EALIGN)])
def test_linear_bwd_refusals(kw, status):
    assert _status("glu_block_linear_bwd", B.LinearBwdArgs, LIN_BWD, kw) == status


def test_workspace_queries():
    n = ctypes.c_size_t(0)
    lib = B._c()
    assert lib.glu_block_norm_bwd_workspace(100, 256, 0, ctypes.byref(n)) == G.GLU_OK and n.value > 0
    assert lib.glu_block_norm_bwd_workspace(100, 256, 3, ctypes.byref(n)) == G.GLU_ESHAPE
    assert lib.glu_block_norm_bwd_workspace(0, 256, 0, ctypes.byref(n)) == G.GLU_EINVAL
    assert lib.glu_block_route_workspace(4, 2, 2000, ctypes.byref(n)) == G.GLU_ESHAPE
    assert lib.glu_block_linear_bwd_workspace(None, ctypes.byref(n)) == G.GLU_EINVAL


def test_valid_calls_without_a_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("checks the no-device status")
    assert _status("glu_block_norm_fwd", B.NormFwdArgs, NORM, {}) == G.GLU_EDEVICE
    assert _status("glu_block_norm_bwd", B.NormBwdArgs, NORM_BWD, {}) == G.GLU_EDEVICE
    assert _status("glu_block_route", B.RouteArgs, ROUTE, {}) == G.GLU_EDEVICE
    assert _status("glu_block_linear_fwd", B.LinearFwdArgs, LIN, {}) == G.GLU_EDEVICE
    assert _status("glu_block_linear_bwd", B.LinearBwdArgs, LIN_BWD, {}) == G.GLU_EDEVICE


def test_tensors_on_the_host_are_refused():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: G.block_norm(x, w_pre=x[0]), lambda: G.route(torch.zeros(2, 2, dtype=torch.int64), 4), lambda: G.linear(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_the_package_is_imported_whole_without_torch():
    """As before there were block operators; they come with torch."""
    r = _python("import sys; sys.modules['torch'] = None\nfrom fp4_quant_gb300 import *\nassert glu_quant_fwd and 'linear' not in dir()")
    assert r.returncode == 0, r.stderr
    r = _python("import sys; sys.modules['torch'] = None\nimport fp4_quant_gb300 as G\nG.linear")
    assert r.returncode != 0 and "torch" in r.stderr
    r = _python("from fp4_quant_gb300 import *\nimport fp4_quant_gb300 as G\nassert linear is G.linear and all(hasattr(G, n) for n in G.__all__)")
    assert r.returncode == 0, r.stderr
