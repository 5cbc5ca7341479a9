"""What the gated activation returns goes into the block operators: its
matrices are contiguous whatever their width, so that rows of a width that is
no multiple of eight do not start on 16 bytes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp4_quant_gb300 as G  # noqa: E402
import test_gpu_block as T  # noqa: E402

BF, F32, DEV = T.BF, T.F32, T.DEV


def _tight(t):
    """The same values, contiguous."""
    return t.clone(memory_format=torch.contiguous_format)


@pytest.mark.parametrize("M,H,D", [(40, 251, 64), (300, 1001, 136), (9, 12, 72)])
def test_linear_fwd_linear_and_back(M, H, D):
    g = T._gen(H)
    x, wg, wu, wd = T._rows(g, M, D), T._rows(g, H, D, scale=D ** -0.5), T._rows(g, H, D, scale=D ** -0.5), T._rows(g, D, H, scale=H ** -0.5)
    gate, up = G.linear(x, wg)["y"], G.linear(x, wu)["y"]
    h = G.fwd(gate, up, act=G.ACT_SILU, fmt=G.FMT_BF16)["out"]
    assert h.is_contiguous() and H % 8 != 0
    y = G.linear(h, wd)["y"]
    S = h.double().abs() @ wd.double().abs().t()
    T._close(y, h.double() @ wd.double().t(), (H + 8) * T.U * S, "y")
    dy = T._rows(g, M, D)
    down = G.linear_bwd(dy, h, wd)
    du = G.bwd(gate, up, down["dx"], act=G.ACT_SILU, fmt=G.FMT_BF16)["out"]  # [M, 2 H]
    both = torch.cat([wg, wu])
    b = G.linear_bwd(du, x, T._rows(g, 2 * H, D).copy_(both), need_db=True)
    d = du.double()
    T._close(b["dx"], d @ both.double(), (2 * H + 8) * T.U * (d.abs() @ both.double().abs()), "dx")
    T._close(b["dw"], d.t() @ x.double(), (M + 8) * T.U * (d.abs().t() @ x.double().abs()), "dw")
    T._close(b["db"], d.sum(0), (M + 8) * T.U * d.abs().sum(0), "db")


@pytest.mark.parametrize("stream", [BF, F32])
def test_every_row_operand_may_be_contiguous(stream):
    g = T._gen(31)
    M, D, K, E, N = 60, 77, 3, 5, 43
    x, b, dy, dr = T._rows(g, M, D, stream), T._rows(g, M, D), T._rows(g, M, D), T._rows(g, M, D, stream)
    w = torch.randn(D, generator=g, device=DEV)
    f = G.block_norm(x, b, w_pre=w, w_post=w)
    kw = dict(rstd_pre=f["rstd_pre"], w_pre=w, rstd_post=f["rstd_post"], w_post=w)
    r = G.route(T._ids(M, K, E, 0.1), E)
    ys, wt = T._rows(g, M * K, D), torch.rand(M, K, generator=g, device=DEV)
    lw, z, res = T._rows(g, N, D), T._rows(g, M, N), T._rows(g, M, N)

    def run(c):
        out = list(G.block_norm(c(x), c(b), w_pre=w, w_post=w).values())
        out += G.block_norm_bwd(c(f["r"]), c(dy), c(dr), branch=c(b), **kw).values()
        out += [G.dispatch(c(b), r), G.combine(c(ys), r, wt, residual=c(b)), G.dispatch_bwd(c(ys), r), *G.combine_bwd(c(b), c(ys), r, wt).values()]
        out += [G.linear(c(b), lw, residual=c(res))["y"]]
        out += G.linear_bwd(c(z), c(b), lw, z=c(res), act=G.ACT_SILU, need_db=True).values()
        return [t for t in out if t is not None]

    side = torch.cuda.Stream()
    want = run(lambda t: t)
    for p, q in zip(run(_tight), want):
        assert torch.equal(p, q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(_tight)
    side.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_weights_have_to_be_laid_out():
    """A weight would be copied at every call: its owner lays it out once."""
    x = torch.zeros(4, 16, dtype=BF, device=DEV)
    with pytest.raises(G.GluQuantError):
        G.linear(x[:, :13], torch.zeros(8, 13, dtype=BF, device=DEV))
