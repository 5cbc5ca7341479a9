"""The block operators on values far from one: the activations and their
derivatives over every bf16 value, and rows of very large and small numbers.

Tolerances are worst-case bounds, as in test_gpu_block.py.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp4_quant_gb300 as G  # noqa: E402
import test_gpu_block as T  # noqa: E402

BF, F32, DEV = T.BF, T.F32, T.DEV


def _every_bf16():
    return torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).to(DEV)


def _column(values):
    """[n, 1], rows on 16 bytes."""
    buf = torch.zeros(values.numel(), 8, dtype=BF, device=DEV)
    buf[:, 0] = values
    return buf[:, :1]


def _same_nan(got, want, what):
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    return ~torch.isnan(want)


def _check_act(name, y, z):
    """act(z) in bf16.  exp has (2 + 1.2 |z|) units in the last place, |z| up to
    88 before act(z) is below 2^-118; the tanh form's argument six roundings, 88
    of 6 * 2^-24 in the exponent; the normal distribution 7.5e-8 of its formula
    and 2^-21 of fp32.  A quotient by 2^126 and more is 0."""
    want = T._act(name, z)
    ok = _same_nan(y, want, name)
    inf = ok & torch.isinf(want)
    assert torch.equal(y[inf].double(), want[inf])
    ok &= ~inf
    y, want, z = y[ok], want[ok], z[ok].double()
    none = torch.zeros_like(want)
    own = {"none": none, "relu": none, "silu": 2.0 ** -15 * want.abs(), "gelu_tanh": 2.0 ** -13 * want.abs(),
           "gelu_erf": torch.where(z.abs() < 16, 2.0 ** -20 * z.abs(), none)}[name]
    T._close(y, want, own + (0.0 if name in ("none", "relu") else 2.0 ** -118), name)


@pytest.mark.parametrize("act", list(T.ACTS))
def test_activations_over_every_bf16(act):
    """In the epilogue of the tiles, of few tokens and of split sums: z is a
    product of one value with 1, so it is every bf16, infinities and NaN too
    (where the formula gives them: act(-inf) is NaN but for ReLU and none)."""
    z = _every_bf16()
    one = torch.ones(1, 8, dtype=BF, device=DEV)[:, :1]
    y = G.linear(_column(z), one, act=T.ACTS[act], keep_z=True)
    _check_act("none", y["z"][:, 0], z)
    _check_act(act, y["y"][:, 0], z)
    _check_act(act, G.linear(one, _column(z), act=T.ACTS[act])["y"][0], z)
    x, w = torch.zeros(17, 4096, dtype=BF, device=DEV), torch.zeros(1024, 4096, dtype=BF, device=DEV)
    x[:, 0] = 1
    for a in range(0, 65536, 1024):
        w[:, 0] = z[a:a + 1024]
        got = G.linear(x, w, act=T.ACTS[act])["y"]
        _check_act(act, got[0], z[a:a + 1024])
        _check_act(act, got[16], z[a:a + 1024])


def _grad(name, z):
    """act'(z) in 64 bits, at infinities its limits."""
    z = z.double()
    c = 2.0 * math.sqrt(2.0 / math.pi)
    if name == "relu":
        return torch.where(z <= 0, 0.0, 1.0).double()  # 1 at NaN too, as the gated activation's
    if name == "none":
        return torch.ones_like(z)
    if name == "gelu_erf":
        g = 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    else:
        u, du = (z, torch.ones_like(z)) if name == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z * z))
        g = (1 + z * du / (1 + torch.exp(u))) / (1 + torch.exp(-u))
    return torch.where(torch.isinf(z), (z > 0).double(), g)


@pytest.mark.parametrize("act", list(T.ACTS))
def test_activation_gradients_over_every_bf16(act):
    """dz = dy act'(z) with dy = 1: in fp32 as db of a single row, in bf16 as dw
    (x = 1), and as dx of one row per value (w = 1)."""
    z = _every_bf16()
    n = z.numel()
    one = torch.ones(1, 8, dtype=BF, device=DEV)[:, :1]
    ones = torch.ones(1, n, dtype=BF, device=DEV)
    zz = z[None] if act != "none" else None
    b = G.linear_bwd(ones, one, _column(ones[0]), z=zz, act=T.ACTS[act], need_dx=False, need_db=True)
    zz = _column(z) if act != "none" else None
    ones = torch.ones(n, 8, dtype=BF, device=DEV)[:, :1]
    dx = G.linear_bwd(ones, ones, one, z=zz, act=T.ACTS[act], need_dw=False)["dx"][:, 0]
    want = _grad(act, z)
    # 2^-18 (1 + |z|) as for values near one; 1 - s is good to three units of
    # 2^-23, which counts |z| u'(z) times; from 16 on act' is 0 or 1
    zc = z.double().abs().clamp(max=16.0)
    own = 2.0 ** -18 * (1 + zc)
    if act == "gelu_tanh":
        own = own + 3 * T.U * zc * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * zc * zc)
    if act in ("none", "relu"):
        own = 0.0 * zc
    for what, got in (("db", b["db"]), ("dw", b["dw"][:, 0]), ("dx", dx)):
        ok = _same_nan(got, want, f"{act} {what}")
        T._close(got[ok], want[ok], torch.nan_to_num(own)[ok], f"{act} {what}")


def test_one_large_z_leaves_the_others_alone():
    """A few large z of tanh-GELU among ordinary ones: dx, dw and db stay the
    formula's (they took NaN from one z of -1e13)."""
    g = T._gen(12)
    M, N, K = 90, 136, 72
    x, w, dy, z = T._rows(g, M, K), T._rows(g, N, K, scale=K ** -0.5), T._rows(g, M, N), T._rows(g, M, N)
    z[3, 7], z[5, 9], z[40, 130], z[41, 0] = -1.5e13, 3e19, -3e38, 3e38
    got = G.linear_bwd(dy, x, w, z=z, act=G.ACT_GELU_TANH, need_db=True)
    dz = dy.double() * _grad("gelu_tanh", z)
    own = dy.double().abs() * 2.0 ** -17 * (1 + z.double().abs().clamp(max=16.0))
    err = own + T.HALF * dz.abs()
    T._close(got["db"], dz.sum(0), own.sum(0) + (M + 8) * T.U * dz.abs().sum(0), "db")
    T._close(got["dx"], dz @ w.double(), ((N + 8) * T.U * dz.abs() + err) @ w.double().abs(), "dx")
    T._close(got["dw"], dz.t() @ x.double(), ((M + 8) * T.U * dz.abs() + err).t() @ x.double().abs(), "dw")


@pytest.mark.parametrize("D", [264, 8192])
@pytest.mark.parametrize("scale", [1e14, 1e-14])
@pytest.mark.parametrize("gates", [1, 160])
def test_norm_backward_of_branches_far_from_one(D, scale, gates):
    """rstd_post^3 is outside fp32's range, the gradients are not."""
    M = 160
    g, r, b, gate, w1, w2 = T._norm_inputs(M, D, BF, F32, True, True, gates, 0.0, D)
    b = (b.double() * scale).to(BF)
    dy, dr = T._rows(g, M, D), T._rows(g, M, D)
    rs = torch.rsqrt(r.float().square().mean(1) + 1e-6)
    rp = torch.rsqrt(b.double().square().mean(1)).float()
    got = G.block_norm_bwd(r, dy, dr, rstd_pre=rs, w_pre=w1, branch=b, rstd_post=rp, w_post=w2, gate=gate)
    want, size = T._norm_bwd_ref(r, dy, dr, rs, w1, b, rp, w2, gate, 1.0, 0.0)
    for k, v in got.items():
        T._close(v, want[k], (2 * D + M + 64) * T.U * size[k], k)
