"""The block operators against their definitions in 64 bits.

Tolerances are worst-case bounds, element by element: u = 2^-23 per operation
along a sum of n terms (n u times the sum of the terms' sizes), which covers
fp32 rounding in any order and the tensor cores' truncation, plus 2^-8 of the
value where it is rounded to bf16 (half a unit in the last of 8 bits).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp4_quant_gb300 as G  # noqa: E402

DEV = torch.device("cuda:0")
U, HALF = 2.0 ** -23, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(g, M, D, dtype=BF, ld=None, scale=1.0):
    """A random matrix with row stride ld (the pad is NaN: nothing may read it)."""
    ld = ld or -(-D // 8) * 8
    buf = torch.full((M, ld), float("nan"), dtype=dtype, device=DEV)
    buf[:, :D] = (scale * torch.randn(M, D, generator=g, device=DEV)).to(dtype)
    return buf[:, :D]


def _close(got, want, slack, what, rounds=None):
    """|got - want| <= slack, + HALF |want| where got is bf16."""
    tol = slack + (HALF * want.abs() if (rounds if rounds is not None else got.dtype is BF) else 0.0) + 1e-37
    bad = (got.double() - want).abs() - tol
    assert not torch.isnan(bad).any() and float(bad.max()) <= 0.0, f"{what}: worst excess {float(bad.max()):.3g}"


# ---- block norms ---------------------------------------------------------------

def _norm_ref(x, branch, w_pre, w_post, gate, alpha, o, eps):
    d = torch.float64
    M, D = x.shape
    r, B, rp = x.to(d), x.to(d).abs(), None
    if branch is not None:
        t = branch.to(d)
        if w_post is not None:
            rp = 1.0 / ((t * t).sum(1) / D + eps).sqrt()
            t = t * rp[:, None] * (w_post.to(d) + o)
        if gate is not None:
            g = gate.to(d).reshape(-1, D)
            t = t * g.repeat_interleave(M // g.shape[0], 0)
        r, B = r + alpha * t, B + abs(alpha) * t.abs()
    rs = 1.0 / ((r * r).sum(1) / D + eps).sqrt()
    y = None if w_pre is None else r * rs[:, None] * (w_pre.to(d) + o)
    return r, y, rs, rp, B


NORM_CASES = [
    # M, D, stream, weights, branch, post, gates, alpha, offset
    (1, 1, BF, BF, True, True, 1, 1.0, 0.0), (1, 4096, BF, BF, True, True, 1, 1.0, 0.0), (3, 7, F32, F32, True, True, 3, 0.5, 1.0),
    (5, 256, BF, BF, False, False, 0, 1.0, 0.0), (12, 1001, F32, BF, True, False, 4, -0.5, 1.0), (700, 264, BF, F32, True, True, 7, 1.0, 1.0),
    (64, 2049, BF, BF, True, False, 0, 1.0, 0.0), (6, 8192, F32, F32, True, True, 2, 0.25, 0.0), (9, 12295, BF, BF, True, True, 1, 1.0, 0.0),
    (400, 4100, F32, BF, True, True, 400, 1.0, 0.0), (2, 16384, F32, F32, True, True, 1, 1.0, 0.0), (1600, 40, BF, BF, True, True, 800, 2.0, 0.0),
]


def _norm_inputs(M, D, stream, wt, branch, post, gates, o, seed):
    g = _gen(seed)
    x = _rows(g, M, D, stream, ld=-(-D // 8) * 8 + 16)
    b = _rows(g, M, D) if branch else None
    gate = _rows(g, gates, D) if gates else None
    w1 = (1.0 - o + 0.1 * torch.randn(D, generator=g, device=DEV)).to(wt)
    w2 = (1.0 - o + 0.1 * torch.randn(D, generator=g, device=DEV)).to(wt) if post else None
    return g, x, b, gate, w1, w2


@pytest.mark.parametrize("M,D,stream,wt,branch,post,gates,alpha,o", NORM_CASES)
def test_norm_forward(M, D, stream, wt, branch, post, gates, alpha, o):
    _, x, b, gate, w1, w2 = _norm_inputs(M, D, stream, wt, branch, post, gates, o, M + D)
    got = G.block_norm(x, b, w_pre=w1, w_post=w2, gate=gate, alpha=alpha, w_offset=o)
    r, y, rs, rp, B = _norm_ref(x, b, w1, w2, gate, alpha, o, 1e-6)
    n = (D + 32) * U
    if branch:
        assert got["r"].dtype is stream
        _close(got["r"], r, n * B, "r")
    else:
        assert got["r"] is None
    grow = ((B * B).sum(1) / (r * r).sum(1)).sqrt()  # of the rounding in r, relative to its norm
    _close(got["rstd_pre"], rs, n * rs * grow, "rstd_pre")
    _close(got["y"], y, n * (rs[:, None] * (w1.double() + o).abs() * B + y.abs() * grow[:, None]), "y")
    if post:
        _close(got["rstd_post"], rp, n * rp, "rstd_post")


def test_norm_forward_without_the_next_norm_and_into_given_outputs():
    _, x, b, gate, _, w2 = _norm_inputs(33, 520, BF, BF, True, True, 1, 0.0, 5)
    full = G.block_norm(x, b, w_post=w2, gate=gate)
    assert full["y"] is None and full["rstd_pre"] is None
    wide = torch.full((33, 1040), -7.0, dtype=BF, device=DEV)
    again = G.block_norm(x, b, w_post=w2, gate=gate[0], out={"r": wide[:, :520]})
    assert again["r"].data_ptr() == wide.data_ptr() and torch.equal(again["r"], full["r"])
    assert bool((wide[:, 520:] == -7.0).all())


def test_norm_rows_of_zeros_and_of_infinities():
    x = torch.zeros(4, 264, dtype=BF, device=DEV)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    w = torch.ones(264, dtype=BF, device=DEV)
    o = G.block_norm(x, w_pre=w, eps=1e-6)
    assert bool((o["y"][0] == 0).all()) and bool((o["y"][3] == 0).all())
    assert abs(float(o["rstd_pre"][0]) - 1e3) < 1e-2
    assert float(o["rstd_pre"][1]) == 0.0 and bool(torch.isnan(o["y"][1, 3])) and bool((o["y"][1, :3] == 0).all())
    assert bool(torch.isnan(o["y"][2]).all())


def _norm_bwd_ref(r, dy, dr, rs, w1, b, rp, w2, gate, alpha, o):
    """The gradients and the sizes of their terms (with every sum over absolute values)."""
    d = torch.float64
    M, D = r.shape
    n, u = r.to(d) * rs.to(d)[:, None], dy.to(d) * (w1.to(d) + o)
    k = rs.to(d)[:, None]
    dR = k * (u - n * ((u * n).sum(1, keepdim=True) / D))
    S = k * (u.abs() + n.abs() * ((u * n).abs().sum(1, keepdim=True) / D))
    if dr is not None:
        dR, S = dR + dr.to(d), S + dr.to(d).abs()
    out, size = {"dx": dR, "dw_pre": (dy.to(d) * n).sum(0)}, {"dx": S, "dw_pre": (dy.to(d) * n).abs().sum(0)}
    if b is None:
        return out, size
    grow = 1.0
    if gate is not None:
        g = gate.to(d).reshape(-1, D)
        grow = g.repeat_interleave(M // g.shape[0], 0)
    down, Sd = alpha * grow * dR, abs(alpha) * (grow.abs() if gate is not None else 1.0) * S
    t = b.to(d)
    if w2 is not None:
        q = rp.to(d)[:, None]
        n2, w = t * q, w2.to(d) + o
        out["dw_post"], size["dw_post"] = (down * n2).sum(0), (Sd * n2.abs()).sum(0)
        t, u, Su = n2 * w, down * w, Sd * w.abs()
        out["dbranch"] = q * (u - n2 * ((u * n2).sum(1, keepdim=True) / D))
        size["dbranch"] = q * (Su + n2.abs() * ((Su * n2.abs()).sum(1, keepdim=True) / D))
    else:
        out["dbranch"], size["dbranch"] = down, Sd
    if gate is not None:
        G_ = g.shape[0]
        out["dgate"] = (alpha * t * dR).reshape(G_, M // G_, D).sum(1)
        size["dgate"] = (abs(alpha) * t.abs() * S).reshape(G_, M // G_, D).sum(1)
    return out, size


@pytest.mark.parametrize("M,D,stream,wt,branch,post,gates,alpha,o", NORM_CASES)
@pytest.mark.parametrize("with_dr", [True, False])
def test_norm_backward(M, D, stream, wt, branch, post, gates, alpha, o, with_dr):
    g, r, b, gate, w1, w2 = _norm_inputs(M, D, stream, wt, branch, post, gates, o, 3 * M + D)
    dy = _rows(g, M, D)
    dr = _rows(g, M, D, stream) if with_dr else None
    rs = torch.rsqrt(r.float().square().mean(1) + 1e-6)
    rp = torch.rsqrt(b.float().square().mean(1) + 1e-6) if post else None
    got = G.block_norm_bwd(r, dy, dr, rstd_pre=rs, w_pre=w1, branch=b, rstd_post=rp, w_post=w2, gate=gate, alpha=alpha, w_offset=o)
    want, size = _norm_bwd_ref(r, dy, dr, rs, w1, b, rp, w2, gate, alpha, o)
    for k, v in got.items():
        assert (v is None) == (k not in want), k
        if v is not None:
            _close(v, want[k], (2 * D + M + 64) * U * size[k], k)


def test_norm_backward_of_the_residual_sum_alone():
    g, x, b, gate, _, w2 = _norm_inputs(30, 200, BF, BF, True, True, 5, 0.0, 11)
    dr = _rows(g, 30, 200)
    rp = torch.rsqrt(b.float().square().mean(1) + 1e-6)
    got = G.block_norm_bwd(x, None, dr, branch=b, rstd_post=rp, w_post=w2, gate=gate)
    assert torch.equal(got["dx"], dr) and got["dw_pre"] is None
    z = torch.zeros(30, 200, dtype=BF, device=DEV)
    want, size = _norm_bwd_ref(z, z, dr, rp, w2, b, rp, w2, gate, 1.0, 0.0)
    for k in ("dbranch", "dw_post", "dgate"):
        _close(got[k], want[k], 600 * U * size[k], k)


@pytest.mark.parametrize("post,gates", [(True, 1), (True, 6), (False, 2), (False, 0)])
def test_norm_gradients_against_differences(post, gates):
    """The gradients' products with a direction against central differences of
    sum(y a + r c) of the 64-bit forward (h^2 of the third derivative: O(1e-8))."""
    M, D, o, alpha = 24, 72, 0.0, 0.75
    g, x, b, gate, w1, w2 = _norm_inputs(M, D, F32, F32, True, post, gates, o, 17)
    a, c = _rows(g, M, D), _rows(g, M, D, F32)
    got = G.block_norm(x, b, w_pre=w1, w_post=w2, gate=gate if gates else None, alpha=alpha)
    grads = G.block_norm_bwd(got["r"], a, c, rstd_pre=got["rstd_pre"], w_pre=w1, branch=b, rstd_post=got["rstd_post"], w_post=w2, gate=gate,
                             alpha=alpha)
    names = {"dx": x, "dbranch": b, "dw_pre": w1, "dw_post": w2, "dgate": gate}
    for k, t in names.items():
        if t is None:
            continue
        v = torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64)
        h, f = 1e-4, []
        for sgn in (h, -h):
            args = {n: (q.double() + sgn * v if n == k else q) if q is not None else None for n, q in names.items()}
            r, y, *_ = _norm_ref(args["dx"], args["dbranch"], args["dw_pre"], args["dw_post"], args["dgate"], alpha, o, 1e-6)
            f.append(float((y * a.double()).sum() + (r * c.double()).sum()))
        slope = (f[0] - f[1]) / (2 * h)
        dot = float((grads[k].double().reshape(t.shape) * v).sum())
        # rounding of the gradient (bf16: HALF, fp32: a few hundred U) at random, 6 sigma, and the h^2 term
        unit = HALF if grads[k].dtype is BF else 400 * U
        tol = 6 * unit * float((grads[k].double().reshape(t.shape) * v).norm()) + 1e-5 * (abs(slope) + float(v.norm()))
        assert abs(slope - dot) <= tol, (k, slope, dot, tol)


# ---- routing -------------------------------------------------------------------

def _route_ref(ids, E):
    lists = [[] for _ in range(E)]
    for j, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            lists[e].append(j)
    src = sum(lists, [])
    slot = torch.full((ids.numel(),), -1, dtype=torch.int32)
    slot[torch.tensor(src, dtype=torch.long)] = torch.arange(len(src), dtype=torch.int32)
    off = torch.tensor([0] + [len(v) for v in lists], dtype=torch.int64).cumsum(0).int()
    return slot.reshape(ids.shape), torch.tensor(src + [-1] * (ids.numel() - len(src)), dtype=torch.int32), off


ROUTES = [(1, 1, 1, 0.0), (1, 8, 128, 0.0), (7, 3, 5, 0.5), (64, 8, 128, 0.0), (1000, 2, 1024, 0.1), (4099, 4, 33, 0.02), (3000, 6, 8, 1.0),
          (20000, 1, 257, 0.3)]


def _ids(T, K, E, drop, dtype=torch.int64, seed=0):
    g = _gen(seed + T)
    ids = (torch.rand(T, K, generator=g, device=DEV).square() * E).to(dtype)  # uneven, some experts empty
    out = torch.rand(T, K, generator=g, device=DEV) < drop
    far = torch.where(torch.rand(T, K, generator=g, device=DEV) < 0.5, -1, E + 5).to(dtype)
    return torch.where(out, far, ids).contiguous()


@pytest.mark.parametrize("T,K,E,drop", ROUTES)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route(T, K, E, drop, dtype):
    ids = _ids(T, K, E, drop, dtype)
    got = G.route(ids, E)
    for k, want in zip(("slot", "src", "offsets"), _route_ref(ids, E)):
        assert torch.equal(got[k].cpu(), want), k


def test_route_takes_wide_ids_as_dropped():
    ids = torch.tensor([[1, 2 ** 32 + 1], [-2 ** 33, 0]], device=DEV)
    assert G.route(ids, 4)["slot"].tolist() == [[1, -1], [-1, 0]]


@pytest.mark.parametrize("T,K,E,drop", ROUTES)
@pytest.mark.parametrize("D", [8, 251, 2056])
def test_rows_there_and_back(T, K, E, drop, D):
    g = _gen(D)
    route = G.route(_ids(T, K, E, drop), E)
    slot, src = route["slot"].long(), route["src"].long()
    x, res, dout = _rows(g, T, D, ld=D // 8 * 8 + 24), _rows(g, T, D), _rows(g, T, D)
    w = torch.rand(T, K, generator=g, device=DEV)
    w[slot < 0] = float("nan")  # a dropped weight does not count
    xs = G.dispatch(x, route)
    want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // K], torch.zeros(1, dtype=BF, device=DEV))
    assert torch.equal(xs, want)
    ys = _rows(g, T * K, D)
    ys[int(route["offsets"][-1]):] = float("nan")  # rows past the last expert's do not count
    rows = torch.where((slot >= 0)[..., None], ys[slot.clamp(min=0)].double(), torch.zeros(1, dtype=torch.float64, device=DEV))
    wd = torch.where(slot >= 0, w, torch.zeros_like(w)).double()
    for weights, residual in ((w, res), (w, None), (None, None)):
        got = G.combine(ys, route, weights, residual=residual)
        f = (rows * (wd if weights is not None else torch.ones_like(wd))[..., None])
        want = f.sum(1) + (residual.double() if residual is not None else 0.0)
        _close(got, want, (K + 4) * U * (f.abs().sum(1) + (residual.double().abs() if residual is not None else 0.0)), "combine")
    assert torch.equal(G.dispatch_bwd(ys, route), G.combine(ys, route))
    b = G.combine_bwd(dout, ys, route, w)
    at = src.clamp(min=0)
    want = torch.where((src >= 0)[:, None], w.reshape(-1)[at].double()[:, None] * dout.double()[at // K], torch.zeros(1, dtype=torch.float64, device=DEV))
    _close(b["dys"], want, 2 * U * want.abs(), "dys")
    f = rows * dout.double()[:, None, :]
    _close(b["dw"], f.sum(2), (D + 8) * U * f.abs().sum(2), "dw")


def test_route_gradients_against_differences():
    """combine is linear in ys and in the weights: differences are exact up to
    the 64-bit sums."""
    g = _gen(3)
    T, K, E, D = 40, 3, 6, 48
    route = G.route(_ids(T, K, E, 0.2), E)
    slot = route["slot"].long()
    ys, dout, w = _rows(g, T * K, D), _rows(g, T, D), torch.rand(T, K, generator=g, device=DEV)

    def loss(y, weights):
        rows = y.double()[slot.clamp(min=0)] * (slot >= 0)[..., None]
        return float(((rows * weights.double()[..., None]).sum(1) * dout.double()).sum())

    b = G.combine_bwd(dout, ys, route, w)
    v = torch.randn(T * K, D, generator=g, device=DEV, dtype=torch.float64)
    slope = (loss(ys.double() + v, w) - loss(ys.double() - v, w)) / 2
    assert abs(slope - float((b["dys"].double() * v).sum())) <= 6 * HALF * float((b["dys"].double() * v).norm()) + 1e-9 * abs(slope)
    v = torch.randn(T, K, generator=g, device=DEV, dtype=torch.float64)
    slope = (loss(ys, w.double() + v) - loss(ys, w.double() - v)) / 2
    assert abs(slope - float((b["dw"].double() * v).sum())) <= 60 * U * float((b["dw"].double().abs() * v.abs()).sum()) + 1e-9 * abs(slope)


# ---- linear --------------------------------------------------------------------

ACTS = {"none": G.ACT_IDENTITY, "silu": G.ACT_SILU, "gelu_tanh": G.ACT_GELU_TANH, "relu": G.ACT_RELU, "gelu_erf": G.ACT_GELU_ERF}


def _act(name, z):
    z = z.double()
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "gelu_erf":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return torch.relu(z) if name == "relu" else z


def _act_grad(name, z):
    z = z.double().clone().requires_grad_(True)
    _act(name, z).sum().backward()
    return z.grad


LINEAR = [
    # M, N, K, act, bias, residual, z
    (1, 1, 1, "none", None, False, False), (1, 1024, 2048, "none", None, True, False), (3, 40, 72, "silu", F32, True, True),
    (16, 257, 1000, "gelu_tanh", BF, False, True), (65, 300, 129, "relu", BF, True, False), (128, 256, 64, "none", None, False, False),
    (129, 513, 320, "gelu_erf", F32, True, True), (300, 1000, 2047, "silu", BF, False, False), (1000, 776, 513, "none", F32, True, False),
    (31, 8192, 512, "gelu_tanh", F32, False, True), (2500, 1100, 200, "none", None, False, False),
]


@pytest.mark.parametrize("M,N,K,act,bias,residual,keep", LINEAR)
def test_linear_forward(M, N, K, act, bias, residual, keep):
    g = _gen(M + N + K)
    x, w = _rows(g, M, K, ld=-(-K // 8) * 8 + 8), _rows(g, N, K, scale=K ** -0.5)
    b = torch.randn(N, generator=g, device=DEV).to(bias) if bias is not None else None
    res = _rows(g, M, N) if residual else None
    got = G.linear(x, w, bias=b, act=ACTS[act], residual=res, keep_z=keep)
    z = x.double() @ w.double().t() + (b.double() if b is not None else 0.0)
    S = x.double().abs() @ w.double().abs().t() + (b.double().abs() if b is not None else 0.0)
    y = _act(act, z) + (res.double() if residual else 0.0)
    # |act'| < 1.2; the activations' own error: 2^-19 of |z| (exponential and quotient approximations)
    slack = 1.2 * (K + 8) * U * S + (2.0 ** -19 * z.abs() if act != "none" else 0.0) + (2 * U * (y.abs() + res.double().abs()) if residual else 0.0)
    _close(got["y"], y, slack, "y")
    assert (got["z"] is None) == (not keep)
    if keep:
        _close(got["z"], z, (K + 8) * U * S, "z")


def _check_linear_bwd(got, dy, x, w, z, act, cuts, need_db=True):
    M, K = x.shape
    N = dy.shape[1]
    f = _act_grad(act, z) if z is not None else torch.ones(1, dtype=torch.float64, device=DEV)
    dz = dy.double() * f
    # dz is rounded to bf16 for the products; act' itself to 2^-18 of (1 + |z|)
    own = dy.double().abs() * (2.0 ** -18 * (1 + z.double().abs())) if z is not None else torch.zeros_like(dz)
    err = own + (HALF * dz.abs() if z is not None else 0.0)
    dx, tx = torch.zeros(M, K, dtype=torch.float64, device=DEV), torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        we = (w[e] if w.dim() == 3 else w).double()
        xe, d, er = x[a:b].double(), dz[a:b], err[a:b]
        dx[a:b] = d @ we
        tx[a:b] = ((N + 8) * U * (d.abs() + er) + er) @ we.abs()
        dw = d.t() @ xe
        tw = ((b - a + 8) * U * (d.abs() + er) + er).t() @ xe.abs()
        _close((got["dw"][e] if w.dim() == 3 else got["dw"]), dw, tw, f"dw[{e}]")
        if need_db:
            _close((got["db"][e] if w.dim() == 3 else got["db"]), d.sum(0), (b - a + 8) * U * d.abs().sum(0) + own[a:b].sum(0), f"db[{e}]")
    _close(got["dx"], dx, tx, "dx")


@pytest.mark.parametrize("M,N,K,act", [(c[0], c[1], c[2], c[3]) for c in LINEAR])
def test_linear_backward(M, N, K, act):
    g = _gen(M * 3 + N + K)
    x, w, dy = _rows(g, M, K, ld=-(-K // 8) * 8 + 8), _rows(g, N, K, scale=K ** -0.5), _rows(g, M, N, ld=-(-N // 8) * 8 + 8)
    z = _rows(g, M, N) if act != "none" else None
    got = G.linear_bwd(dy, x, w, z=z, act=ACTS[act], need_db=True)
    _check_linear_bwd(got, dy, x, w, z, act, [0, M])
    if z is not None:  # the sums alone, without a product that takes dz
        only = G.linear_bwd(dy, x, w, z=z, act=ACTS[act], need_dx=False, need_dw=False, need_db=True)
        assert only["dx"] is None and only["dw"] is None and torch.equal(only["db"], got["db"])


EXPERTS = [
    # rows per expert, rows past the last, N, K, act
    ([1], 0, 64, 64, "none"), ([0, 3, 0, 0, 130, 1], 4, 300, 200, "silu"), ([64, 128, 256], 0, 512, 256, "none"),
    ([5, 0, 77, 63, 65, 1, 0], 9, 129, 73, "gelu_tanh"), ([0, 0], 20, 72, 40, "relu"), ([300, 1, 513], 1, 264, 1030, "gelu_erf"),
    ([1] * 40, 0, 256, 512, "none"), ([2, 0] * 200 + [700], 3, 80, 88, "silu"),
]


@pytest.mark.parametrize("counts,spare,N,K,act", EXPERTS)
def test_linear_by_expert(counts, spare, N, K, act):
    E, cuts = len(counts), [0]
    for n in counts:
        cuts.append(cuts[-1] + n)
    M = cuts[-1] + spare
    g = _gen(M + N + K)
    x, dy, res, z = _rows(g, M, K), _rows(g, M, N), _rows(g, M, N), _rows(g, M, N)
    w = torch.full((E, N, -(-K // 8) * 8 + 8), float("nan"), dtype=BF, device=DEV)[:, :, :K]
    w[:] = (K ** -0.5 * torch.randn(E, N, K, generator=g, device=DEV)).to(BF)
    bias = torch.randn(E, N, generator=g, device=DEV)
    off = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    if spare:  # what lies past the last expert's rows does not count
        for t in (x, dy, res, z):
            t[cuts[-1]:] = float("nan")
    got = G.linear(x, w, bias=bias, act=ACTS[act], residual=res, offsets=off, keep_z=True)
    for k in ("y", "z"):
        assert bool((got[k][cuts[-1]:] == 0).all()), k
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        zz = x[a:b].double() @ w[e].double().t() + bias[e].double()
        S = x[a:b].double().abs() @ w[e].double().abs().t() + bias[e].double().abs()
        y = _act(act, zz) + res[a:b].double()
        if a < b:
            _close(got["z"][a:b], zz, (K + 8) * U * S, f"z[{e}]")
            _close(got["y"][a:b], y, 1.2 * (K + 8) * U * S + (2.0 ** -19 * zz.abs() if act != "none" else 0.0)
                   + 2 * U * (y.abs() + res[a:b].double().abs()), f"y[{e}]")
    zb = z if act != "none" else None
    b = G.linear_bwd(dy, x, w, z=zb, act=ACTS[act], offsets=off, need_db=True)
    zeroed = [t.clone() if t is not None else None for t in (dy, x, zb)]
    for t in zeroed:
        if t is not None:
            t[cuts[-1]:] = 0
    _check_linear_bwd(b, zeroed[0], zeroed[1], w, zeroed[2], act, cuts)


def test_an_expert_does_not_see_its_neighbours_nan():
    """dw sums over one expert's rows only, whatever the next one's hold."""
    g = _gen(9)
    cuts = [0, 70, 140, 141]
    x, dy = _rows(g, 141, 96), _rows(g, 141, 72)
    x[70:140], dy[70:140] = float("inf"), float("nan")
    w = (0.1 * torch.randn(3, 72, 96, generator=g, device=DEV)).to(BF)
    w[1] = float("nan")
    off = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    b = G.linear_bwd(dy, x, w, offsets=off, need_db=True)
    for e, (p, q) in ((0, (0, 70)), (2, (140, 141))):
        d, xe = dy[p:q].double(), x[p:q].double()
        _close(b["dw"][e], d.t() @ xe, 80 * U * (d.abs().t() @ xe.abs()), "dw")
        _close(b["dx"][p:q], d @ w[e].double(), 80 * U * (d.abs() @ w[e].double().abs()), "dx")
        _close(b["db"][e], d.sum(0), 80 * U * d.abs().sum(0), "db")
    y = G.linear(x, w, offsets=off)["y"]
    assert bool(torch.isfinite(y[:70]).all()) and bool(torch.isfinite(y[140:]).all())


@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh", "gelu_erf"])
def test_linear_gradients_against_differences(act):
    M, N, K = 24, 40, 56
    g = _gen(21)
    x, w, dy = _rows(g, M, K), _rows(g, N, K, scale=K ** -0.5), _rows(g, M, N)
    bias = torch.randn(N, generator=g, device=DEV)
    z = G.linear(x, w, bias=bias, act=ACTS[act], keep_z=True)["z"]
    b = G.linear_bwd(dy, x, w, z=z if act != "none" else None, act=ACTS[act], need_db=True)
    for k, t in (("dx", x), ("dw", w), ("db", bias)):
        v = torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64)
        h, f = 1e-4, []
        for s in (h, -h):
            q = {n: (a.double() + s * v if n == k else a.double()) for n, a in (("dx", x), ("dw", w), ("db", bias))}
            f.append(float((_act(act, q["dx"] @ q["dw"].t() + q["db"]) * dy.double()).sum()))
        slope, dot = (f[0] - f[1]) / (2 * h), float((b[k].double() * v).sum())
        # the gradient is taken at z rounded to bf16 (|act''| < 1.2: HALF |z| of it) and holds a rounded dz
        sens = {"dx": dy.double().abs() @ w.double().abs(), "dw": dy.double().abs().t() @ x.double().abs(), "db": dy.double().abs().sum(0)}[k]
        tol = 6 * HALF * (1 + 1.2 * float(z.double().abs().mean())) * float((sens * v.abs()).norm()) + 1e-6 * abs(slope)
        assert abs(slope - dot) <= tol, (k, slope, dot, tol)


# ---- addressing, streams, repeats ------------------------------------------------

def test_offsets_beyond_32_bits():
    """Rows 2^30 elements apart: byte and element offsets pass 2^32 and 2^31."""
    ld, D, M = 1 << 30, 72, 4
    g = _gen(2)
    buf = torch.empty(3 * ld + D, dtype=BF, device=DEV)
    x = buf.as_strided((M, D), (ld, 1))
    x.copy_(torch.randn(M, D, generator=g, device=DEV).to(BF))
    small = x.contiguous()
    w = torch.ones(D, dtype=BF, device=DEV)
    assert torch.equal(G.block_norm(x, small, w_pre=w)["y"], G.block_norm(small, small, w_pre=w)["y"])
    wt = _rows(g, 40, D)
    assert torch.equal(G.linear(x, wt)["y"], G.linear(small, wt)["y"])
    route = G.route(torch.tensor([[1], [0], [-1], [1]], device=DEV), 2)
    assert torch.equal(G.dispatch(x, route), G.dispatch(small, route))
    out = buf.as_strided((M, D), (ld, 1))
    keep = G.combine(small, route)
    G.combine(small, route, out=out)
    assert torch.equal(out, keep)
    dy = _rows(g, M, 40)
    a, b = G.linear_bwd(dy, x, wt), G.linear_bwd(dy, out.contiguous(), wt)
    assert torch.equal(a["dw"], b["dw"])


def test_calls_on_another_stream_and_in_a_graph():
    g = _gen(4)
    M, D, N = 300, 512, 640
    x, b, w = _rows(g, M, D), _rows(g, M, D), _rows(g, N, D)
    wn = torch.ones(D, dtype=BF, device=DEV)
    ids = _ids(M, 2, 9, 0.1)

    def work():
        o = G.block_norm(x, b, w_pre=wn, w_post=wn)
        gr = G.block_norm_bwd(o["r"], b, x, rstd_pre=o["rstd_pre"], w_pre=wn, branch=b, rstd_post=o["rstd_post"], w_post=wn)
        r = G.route(ids, 9)
        return [o["y"], gr["dx"], gr["dw_pre"], G.dispatch(o["y"], r), G.linear(o["y"], w, act=G.ACT_SILU)["y"]]

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        o = G.block_norm(x, b, w_pre=wn, w_post=wn, stream=handle)
        gr = G.block_norm_bwd(o["r"], b, x, rstd_pre=o["rstd_pre"], w_pre=wn, branch=b, rstd_post=o["rstd_post"], w_post=wn, stream=handle)
        y = G.linear(o["y"], w, act=G.ACT_SILU, stream=handle)["y"]
        side.synchronize()
        assert torch.equal(o["y"], want[0]) and torch.equal(gr["dx"], want[1]) and torch.equal(gr["dw_pre"], want[2]) and torch.equal(y, want[4])
    with torch.cuda.stream(side):
        for _ in range(2):
            work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_the_same_call_gives_the_same_bits():
    g = _gen(6)
    M, D, N = 1111, 520, 1000
    x, b, dy, w = _rows(g, M, D), _rows(g, M, D), _rows(g, M, D), _rows(g, N, D)
    z, dyn = _rows(g, M, N), _rows(g, M, N)
    wn, rs = torch.ones(D, device=DEV), torch.ones(M, device=DEV)
    runs = [(G.block_norm_bwd(x, dy, b, rstd_pre=rs, w_pre=wn, branch=b, rstd_post=rs, w_post=wn, gate=x[:11]),
             G.linear_bwd(dyn, x, w, z=z, act=G.ACT_SILU, need_db=True)) for _ in range(3)]
    for r in runs[1:]:
        for p, q in zip(runs[0], r):
            assert all(torch.equal(p[k], q[k]) for k in p)


def test_refused_tensors():
    x = torch.zeros(4, 16, dtype=BF, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    r = G.route(ids, 2)
    w = torch.zeros(8, 16, dtype=BF, device=DEV)
    for err, call in [
            (TypeError, lambda: G.block_norm(x.half(), w_pre=x[0])), (ValueError, lambda: G.block_norm(x, x[:2], w_pre=x[0])),
            (ValueError, lambda: G.block_norm(x, w_pre=x[0, :8])), (G.GluQuantError, lambda: G.block_norm(x)),
            (G.GluQuantError, lambda: G.block_norm(x, x, gate=x[:3])), (G.GluQuantError, lambda: G.block_norm(x[:, 1:9], w_pre=x[0, :8])),
            (ValueError, lambda: G.block_norm(x.t(), w_pre=x[:, 0].contiguous())), (TypeError, lambda: G.route(ids.float(), 2)),
            (G.GluQuantError, lambda: G.route(ids, 0)), (ValueError, lambda: G.dispatch(x[:3], r)),
            (ValueError, lambda: G.combine(x, r)), (TypeError, lambda: G.combine(G.dispatch(x, r), r, torch.zeros(4, 2, dtype=BF, device=DEV))),
            (ValueError, lambda: G.linear(x, w[:, :8])), (ValueError, lambda: G.linear(x, w, offsets=r["offsets"])),
            (ValueError, lambda: G.linear(x, w[None])), (G.GluQuantError, lambda: G.linear(x, w, act=G.ACT_BF16_STEPS)),
            (G.GluQuantError, lambda: G.linear_bwd(x[:, :8], x, w, act=G.ACT_SILU)),
            (ValueError, lambda: G.linear(x, w, out={"y": x}))]:
        with pytest.raises(err):
            call()


def test_no_wait_gave_up():
    torch.cuda.synchronize()
    assert G.block_device_errors() == (G.GLU_OK, 0)


# ---- further shapes: rows through the ring, split sums, many experts -------------

@pytest.mark.parametrize("M,D,stream,wt,branch,post,gates,alpha,o", [
    (1000, 1032, BF, BF, True, True, 4, 1.0, 0.0), (611, 2056, F32, F32, True, True, 1, 0.5, 1.0), (640, 4096, BF, F32, True, False, 0, 1.0, 0.0),
    (2000, 515, F32, BF, False, False, 0, 1.0, 0.0), (310, 20000, F32, BF, True, True, 310, 1.0, 1.0), (500, 8192, BF, BF, True, True, 125, 1.0, 0.0)])
def test_norm_rows_through_the_ring(M, D, stream, wt, branch, post, gates, alpha, o):
    test_norm_forward(M, D, stream, wt, branch, post, gates, alpha, o)
    if D <= 16384:
        test_norm_backward(M, D, stream, wt, branch, post, gates, alpha, o, True)


@pytest.mark.parametrize("M,N,K,act,bias,residual,keep", [
    (9, 520, 4096, "silu", BF, True, True), (16, 16400, 264, "gelu_erf", F32, True, False), (17, 600, 2048, "gelu_tanh", F32, True, True),
    (40, 1001, 4103, "relu", BF, True, True), (200, 2048, 1536, "none", None, True, False), (600, 3001, 1032, "silu", F32, False, True)])
def test_linear_of_few_rows(M, N, K, act, bias, residual, keep):
    test_linear_forward(M, N, K, act, bias, residual, keep)
    test_linear_backward(M, N, K, act)


def test_linear_with_the_most_experts():
    test_linear_by_expert([3, 0, 17, 1] * 256, 2, 136, 72, "silu")


def test_rows_of_many_choices():
    """More than eight choices per token, and more than one block of the sort."""
    test_rows_there_and_back(700, 11, 24, 0.1, 264)


def test_results_belong_to_the_given_stream():
    """Memory that a call allocates comes from the pool of the stream it runs
    on: what the current stream still uses cannot be handed out to it."""
    side = torch.cuda.Stream()
    x = torch.ones(64, 512, dtype=BF, device=DEV)
    w = torch.ones(512, dtype=BF, device=DEV)
    torch.cuda.synchronize()
    big = torch.empty(64, 512, dtype=BF, device=DEV)
    at = big.data_ptr()
    torch.cuda._sleep(2_000_000)  # the current stream is busy (about a millisecond) and then writes to big
    big.fill_(-3.0)
    del big  # free for the current stream's next allocation only
    y = G.block_norm(x, w_pre=w, stream=side)["y"]
    assert y.data_ptr() != at
    torch.cuda.synchronize()
    assert bool((y == 1).all())


@pytest.mark.parametrize("D", [5, 517, 1031, 4606])
@pytest.mark.parametrize("stream", [BF, F32])
def test_what_stands_behind_a_row_does_not_count(D, stream):
    """The same bits whatever stands between a row's end and the next row, and
    nothing is written there."""
    T, K, E = 700, 3, 5
    ld = -(-D // 8) * 8

    def run(behind):
        g = _gen(7)

        def rows(M, dtype=BF):
            buf = torch.full((M, ld), behind, dtype=dtype, device=DEV)
            buf[:, :D] = torch.randn(M, D, generator=g, device=DEV).to(dtype)
            return buf[:, :D]

        x, b, dy, dr = rows(T, stream), rows(T), rows(T), rows(T, stream)
        w = torch.randn(D, generator=g, device=DEV)
        got = []
        for gates in (1, 28, T):
            gate = rows(gates)
            r = torch.full((T, ld), 7.0, dtype=stream, device=DEV)
            f = G.block_norm(x, b, w_pre=w, w_post=w, gate=gate, out={"r": r[:, :D]})
            assert bool((r[:, D:] == 7).all())
            r[:, D:] = behind
            back = G.block_norm_bwd(f["r"], dy, dr, rstd_pre=f["rstd_pre"], w_pre=w, branch=b, rstd_post=f["rstd_post"], w_post=w, gate=gate)
            got += [f["r"].clone(), f["y"], *(back[k] for k in ("dx", "dbranch", "dw_pre", "dw_post", "dgate"))]
        tok, ys, wt = rows(T), rows(T * K), torch.rand(T, K, generator=g, device=DEV)
        ids = torch.randint(-1, E, (T, K), generator=g, device=DEV, dtype=torch.int32)
        ids[0] = torch.tensor([E - 1] * K)
        at = G.route(ids, E)
        out = torch.full((T, ld), 7.0, dtype=BF, device=DEV)
        got.append(G.combine(ys, at, wt, residual=tok, out=out[:, :D]).clone())
        assert bool((out[:, D:] == 7).all())
        back = G.combine_bwd(tok, ys, at, wt)
        got += [G.dispatch(tok, at), back["dys"], back["dw"]]
        lin = G.linear_bwd(tok, rows(T), rows(D), z=rows(T), act=G.ACT_SILU, need_db=True)
        return got + [lin[k] for k in ("dx", "dw", "db")]

    want = run(0.0)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for behind in (float("nan"), float("inf")):
        for i, (a, t) in enumerate(zip(want, run(behind))):
            assert torch.equal(a, t), (behind, i)
