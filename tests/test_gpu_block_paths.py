"""Paths of the block operators that only some shapes take: wide norms with
several rows per block, split sums on a side stream, experts in a graph, the
accumulators' hand-over between the CTAs of a pair."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp4_quant_gb300 as G  # noqa: E402
import test_gpu_block as T  # noqa: E402

BF, F32, DEV = T.BF, T.F32, T.DEV


# Many more rows than blocks (at most one per SM here) times stages: every
# stage is refilled several times, and the sums over rows are carried along.
# One stage of the backward: fp32 rows above 9600 wide, or 8228 with a gate row
# per few rows; bf16 above 14400 and 11520.
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("M,D,gates", [(1400, 8200, 1), (1400, 12288, 1), (1400, 12288, 700), (1100, 12295, 1), (1100, 12295, 550), (1000, 16384, 1),
                                       (1000, 16384, 500), (900, 16377, 900)])
def test_wide_norms_of_many_rows(M, D, gates, stream):
    args = (M, D, stream, F32 if stream is BF else BF, True, True, gates, 0.5, 1.0)
    T.test_norm_forward(*args)
    T.test_norm_backward(*args, True)


@pytest.mark.parametrize("M,D,stream", [(700, 16392, F32), (900, 32768, BF), (500, 32761, F32)])
def test_widest_norms_forward(M, D, stream):
    T.test_norm_forward(M, D, stream, BF, True, True, 1, 1.0, 0.0)


@pytest.mark.parametrize("M,D,stream", [(1000, 16384, F32), (1000, 12288, BF)])
def test_wide_norms_without_a_branch_and_without_dr(M, D, stream):
    T.test_norm_forward(M, D, stream, BF, False, False, 0, 1.0, 0.0)
    T.test_norm_backward(M, D, stream, BF, False, False, 0, 1.0, 0.0, False)


def test_wide_norms_give_the_same_bits():
    g = T._gen(8)
    M, D = 1000, 16384
    x, b, dy, dr = T._rows(g, M, D, F32), T._rows(g, M, D), T._rows(g, M, D), T._rows(g, M, D, F32)
    w, rs = torch.ones(D, device=DEV), torch.ones(M, device=DEV)
    for gate in (T._rows(g, 1, D), T._rows(g, 500, D)):
        runs = [G.block_norm_bwd(x, dy, dr, rstd_pre=rs, w_pre=w, branch=b, rstd_post=rs, w_post=w, gate=gate) for _ in range(4)]
        for r in runs[1:]:
            assert all(torch.equal(runs[0][k], r[k]) for k in r)


def test_split_sums_on_a_side_stream_and_experts_in_a_graph():
    g = T._gen(14)
    x, w, dy = T._rows(g, 40, 4096), T._rows(g, 520, 4096), T._rows(g, 40, 520)
    z = T._rows(g, 40, 520)
    cuts = torch.tensor([0, 70, 70, 201, 290], dtype=torch.int32, device=DEV)
    xe, dye, ze = T._rows(g, 300, 264), T._rows(g, 300, 136), T._rows(g, 300, 136)
    we, bias = T._rows(g, 4 * 136, 264).reshape(4, 136, 264), torch.randn(4, 136, generator=g, device=DEV)
    ids = T._ids(300, 2, 9, 0.1)
    wt = torch.rand(300, 2, generator=g, device=DEV)

    def work(stream=None):
        y = G.linear(x, w, act=G.ACT_SILU, residual=dy, keep_z=True, stream=stream)
        b = G.linear_bwd(dy, x, w, z=z, act=G.ACT_SILU, need_db=True, stream=stream)
        e = G.linear(xe, we, bias=bias, act=G.ACT_GELU_ERF, offsets=cuts, keep_z=True, stream=stream)
        f = G.linear_bwd(dye, xe, we, z=ze, act=G.ACT_GELU_ERF, offsets=cuts, need_db=True, stream=stream)
        r = G.route(ids, 9, stream=stream)
        s = G.dispatch(xe, r, stream=stream)
        c = G.combine_bwd(xe, s, r, wt, stream=stream)
        return [y["y"], y["z"], *b.values(), e["y"], e["z"], *f.values(), s, G.combine(s, r, wt, residual=xe, stream=stream), *c.values()]

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = work(handle)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


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
