"""Paths of the block operators that only some shapes take: the accumulators'
hand-over between the CTAs of a pair."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp4_quant_gb300 as G  # noqa: E402
import test_gpu_block as T  # noqa: E402

BF, F32, DEV = T.BF, T.F32, T.DEV


@pytest.mark.parametrize("M,N,K", [(20000, 1000, 64), (9000, 2500, 40)])
def test_accumulators_handed_over_between_the_ctas(M, N, K):
    """Sums of one slice each: the products wait for the epilogue's reads of both
    CTAs at every tile, and an early one would overwrite what is being read."""
    g = T._gen(M)
    x, w, dy, b = T._rows(g, M, K), T._rows(g, N, K), T._rows(g, M, N), torch.randn(N, generator=g, device=DEV)
    want = x.double() @ w.double().t() + b.double()
    size = x.double().abs() @ w.double().abs().t() + b.double().abs()
    first = None
    for _ in range(6):
        y = G.linear(x, w, bias=b, keep_z=True)
        T._close(y["y"], want, (K + 8) * T.U * size, "y")
        T._close(y["z"], want, (K + 8) * T.U * size, "z")
        if first is None:
            first = y["y"]
        assert torch.equal(first, y["y"])
    assert torch.equal(G.linear_bwd(dy, x, w)["dw"], G.linear_bwd(dy, x, w)["dw"])
