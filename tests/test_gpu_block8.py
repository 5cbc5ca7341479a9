"""The operators in 8 bits against their definitions in 64 bits.

Tolerances are worst-case bounds, element by element.  Codes and scales of bf16
values are exact.  Codes of fp32 results are those of a value within the result's
error bound of the definition's, with a block maximum within its largest one, and
2^-22 for the quotient.  Sums: U = 2^-23 per operation along a sum of n terms (n U
times the sum of the terms' sizes), which covers fp32 rounding in any order and the
tensor cores' truncation, plus 2^-8 of the value where it is rounded to bf16 (half
a unit in the last of 8 bits).  The activations' bounds are derived in _act_err.
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
TOP, LEAST = 448.0, 2.0 ** -100
F8, BF, F32, F64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.float64
ACTS = [G.ACT_SILU, G.ACT_GELU_TANH, G.ACT_RELU, G.ACT_IDENTITY, G.ACT_GELU_ERF]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _padded(values, dtype, pad=8):
    n = values.shape[-1]
    buf = torch.zeros(*values.shape[:-1], -(-n // pad) * pad, dtype=dtype, device=DEV)[..., :n]
    return buf.copy_(values)


def _x(M, K, seed, scale=1.0):
    g = _gen(seed)
    v = torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(M, 1, generator=g, device=DEV)) * scale
    return _padded(v, BF)


def _offsets(M, E, seed, spare=0, empty=()):
    """Random cuts of M - spare rows among E experts, some of them without rows."""
    p = torch.rand(E, generator=_gen(seed), device=DEV, dtype=F64).cpu() + 0.05
    for e in empty:
        p[e] = 0
    ends = (torch.cumsum(p, 0) / p.sum() * (M - spare)).round().long()
    return torch.tensor([0] + ends.tolist(), dtype=torch.int32, device=DEV)


def _power(e):
    """2^e in fp64, from its bits (on a GPU ldexp is a product with an fp32 power, which may be off)."""
    return ((e.long() + 1023) << 52).view(F64)


def _e4m3(v):
    """The nearest E4M3 value, ties to even."""
    step = _power((torch.frexp(v)[1] - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _tile(v, rows, cols):
    """Maxima of the blocks of rows x cols, spread over their elements, and as they are."""
    R, C = v.shape
    p = v.new_zeros(-(-R // rows) * rows, -(-C // cols) * cols)
    p[:R, :C] = v
    a = p.view(-1, rows, p.shape[1] // cols, cols).abs().amax((1, 3)).clamp_min(LEAST)
    return a.repeat_interleave(rows, 0)[:R].repeat_interleave(cols, 1)[:, :C], a


def _cols(v, offsets):
    """The rows laid out by column blocks."""
    M = v.shape[0]
    if offsets is None:
        return torch.cat([v, v.new_zeros(-M % 128, v.shape[1])])
    cuts = offsets.tolist()
    E = len(cuts) - 1
    p = v.new_zeros((M // 128 + E) * 128, v.shape[1])
    for e in range(E):
        b = (cuts[e] // 128 + e) * 128
        p[b:b + cuts[e + 1] - cuts[e]] = v[cuts[e]:cuts[e + 1]]
    return p


def _same_bits(got, want):
    assert torch.equal(got.view(torch.uint8) if got.dtype is F8 else got, want.view(torch.uint8) if want.dtype is F8 else want)


def _check_exact(q, s, v, rows, cols, transposed):
    """Codes and scales of bf16 values v (as fp64): the exact ones."""
    spread, a = _tile(v, rows, cols)
    want = (a / TOP).to(F32)  # in fp64: a division of fp32 tensors by a number is a product with its reciprocal
    assert torch.equal(s, want.t() if transposed else want)
    assert torch.equal(q.to(F64), _e4m3(v * TOP / spread))


def _check_near(q, s, v, err, rows, cols, transposed):
    """Codes and scales of values within err (a tensor) of v."""
    spread, a = _tile(v, rows, cols)
    worst, e = _tile(err, rows, cols)
    want = a / TOP
    off = (e + a * 2.0 ** -23) / TOP
    want, off = (want.t(), off.t()) if transposed else (want, off)
    assert bool(((s.to(F64) - want).abs() <= off).all())
    t = v * TOP / spread
    d = err * TOP / spread + t.abs() * (worst / spread + 2.0 ** -22)
    q = q.to(F64)
    bad = (q < _e4m3(t - d)) | (q > _e4m3(t + d))
    assert not bool(bad.any()), (int(bad.sum()), t[bad][:4], q[bad][:4])


SIZES = [(1, 1), (1, 128), (3, 7), (17, 40), (128, 128), (127, 129), (129, 255), (300, 1000), (1000, 16), (257, 2049)]


@pytest.mark.parametrize("M,K", SIZES)
def test_quant_rows_and_columns(M, K):
    x = _x(M, K, M + K)
    v = x.to(F64)
    both = G.quant8(x, rows=True, cols=True)
    _check_exact(both["q"], both["s"], v, 1, 128, True)
    _check_exact(both["qc"], both["sc"], _cols(v, None), 128, 1, False)
    rows, cols = G.quant8(x), G.quant8(x, rows=False, cols=True)
    assert rows["qc"] is None and cols["q"] is None
    for one in (rows, cols):
        for k, t in one.items():
            if t is not None:
                _same_bits(t, both[k])


@pytest.mark.parametrize("M,K,E,spare,empty", [(1, 64, 4, 0, ()), (5, 136, 64, 0, (3, 4)), (300, 200, 3, 20, (0,)), (1000, 264, 7, 300, (2, 6)),
                                               (640, 128, 5, 0, ()), (2000, 130, 1, 1999, ()), (512, 96, 1024, 100, (0, 500, 1023)),
                                               (900, 128, 40, 900, ()), (700, 128, 33, 5, (31, 32))])
def test_quant_by_expert(M, K, E, spare, empty):
    x = _x(M, K, M + E)
    off = _offsets(M, E, M, spare, empty)
    v = x.to(F64)
    o = G.quant8(x, rows=True, cols=True, offsets=off)
    _check_exact(o["q"], o["s"], v, 1, 128, True)
    _check_exact(o["qc"], o["sc"], _cols(v, off), 128, 1, False)
    c = G.quant8(x, rows=False, cols=True, offsets=off)
    _same_bits(c["qc"], o["qc"])
    _same_bits(c["sc"], o["sc"])


@pytest.mark.parametrize("N,K,E", [(1, 1, 0), (128, 128, 0), (130, 70, 0), (256, 384, 3), (40, 1000, 2), (300, 129, 1)])
def test_quant_weight(N, K, E):
    w = _padded(torch.randn(max(E, 1) * N, K, generator=_gen(N), device=DEV), BF)
    if E:
        w = w.view(E, N, K) if K % 8 == 0 else torch.stack([w[e * N:(e + 1) * N] for e in range(E)])
        if K % 8:
            w = _padded(w, BF)
    o = G.quant8_weight(w)
    for e in range(max(E, 1)):
        q, s, v = (o["q"][e], o["s"][e], w[e]) if E else (o["q"], o["s"], w)
        _check_exact(q, s, v.to(F64), 128, 128, False)


def test_every_quotient_of_bf16_mantissas():
    """Rows of one maximum each, against every mantissa at every exponent down to the
    least code: midpoints among them, which go to the even code."""
    m = torch.arange(128, dtype=F64, device=DEV)
    a = (1 + m / 128)[:, None, None]
    e = torch.arange(20, dtype=F64, device=DEV)[None, :, None]
    v = (1 + m / 128)[None, None, :] * _power(-e)
    v = torch.minimum(v.expand(128, 20, 128), a).clone()
    v[:, :, 0] = a[:, :, 0]
    v[:, 1::2] *= -1
    v = v.reshape(-1, 128)
    x = v.to(BF)
    assert torch.equal(x.to(F64), v)
    o = G.quant8(x)
    _check_exact(o["q"], o["s"], v, 1, 128, True)
    t = v * TOP / _tile(v, 1, 128)[0]
    half = _power((torch.frexp(t)[1] - 1).clamp_min(-6) - 4)
    odd = (t.abs() / half) % 2 == 1
    assert int(odd.sum()) > 1000  # there were midpoints
    # the same values down the columns, and through 128 x 128 blocks of one maximum
    c = G.quant8(x.t().contiguous(), rows=False, cols=True)
    _same_bits(c["qc"].t().contiguous(), o["q"].contiguous())
    wq = G.quant8_weight(x[:20].contiguous())
    _check_exact(wq["q"], wq["s"], v[:20], 128, 128, False)


@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -110, 2.0 ** -99, 2.0 ** 120])
def test_quant_of_small_and_large_values(scale):
    x = (torch.randn(130, 256, generator=_gen(5), device=DEV).clamp(-4, 4) * scale).to(BF)
    o = G.quant8(x, rows=True, cols=True)
    v = x.to(F64)
    assert bool(torch.isfinite(o["s"]).all())
    _check_exact(o["q"], o["s"], v, 1, 128, True)
    _check_exact(o["qc"], o["sc"], _cols(v, None), 128, 1, False)
    top = torch.full((128, 128), torch.finfo(BF).max, dtype=BF, device=DEV)
    o = G.quant8(top, rows=True, cols=True)
    assert bool((o["q"].float() == TOP).all()) and bool((o["qc"].float() == TOP).all())
    assert bool(torch.isfinite(o["q"].float() * o["s"].t().repeat_interleave(128, 1)).all())


def test_zeros_keep_their_sign_and_nan_and_infinity_fill_their_block():
    x = _x(200, 300, 9)
    x[3] = 0.0
    x[4] = -0.0
    x[7, 130] = float("nan")
    x[150, 5] = float("inf")
    x[151, 299] = float("-inf")
    o = G.quant8(x, rows=True, cols=True)
    assert bool((o["q"][3].view(torch.uint8) == 0).all()) and bool((o["q"][4].view(torch.uint8) == 0x80).all())
    bad_rows = torch.zeros(200, 3, dtype=torch.bool, device=DEV)
    bad_rows[7, 1] = bad_rows[150, 0] = bad_rows[151, 2] = True
    assert torch.equal(torch.isnan(o["s"].t()), bad_rows)
    assert torch.equal(torch.isnan(o["q"].float()), bad_rows.repeat_interleave(128, 1)[:, :300])
    bad_cols = torch.zeros(2, 300, dtype=torch.bool, device=DEV)
    bad_cols[0, 130] = bad_cols[1, 5] = bad_cols[1, 299] = True
    assert torch.equal(torch.isnan(o["sc"]), bad_cols)
    assert torch.equal(torch.isnan(o["qc"].float()), bad_cols.repeat_interleave(128, 0))
    good = x.to(F64)
    good[7], good[150], good[151] = 0, 0, 0
    spread, _ = _tile(good, 1, 128)
    keep = ~bad_rows.repeat_interleave(128, 1)[:, :300]
    keep[[7, 150, 151]] = False
    assert torch.equal(o["q"].to(F64)[keep], _e4m3(good * TOP / spread)[keep])
    w = G.quant8_weight(x)
    assert torch.equal(torch.isnan(w["s"]), torch.tensor([[False, True, False], [True, False, True]], device=DEV))
    # what a row form keeps of them
    k = G.quant8({"q": o["q"], "s": o["s"]}, rows=False, cols=True)
    cols = bad_rows.repeat_interleave(128, 1)[:, :300]
    assert torch.equal(torch.isnan(k["sc"]), torch.stack([cols[:128].any(0), cols[128:].any(0)]))


def _kept(o):
    q = o["q"].to(F64)
    return q * o["s"].to(F64).t().repeat_interleave(128, 1)[:, :q.shape[1]]


@pytest.mark.parametrize("M,K,E,spare", [(1, 1, 0, 0), (130, 257, 0, 0), (1000, 300, 0, 0), (500, 384, 6, 50), (77, 128, 20, 0)])
def test_kept_rows_as_columns(M, K, E, spare):
    x = G.quant8(_x(M, K, M))
    off = _offsets(M, E, K, spare, (1,)) if E else None
    o = G.quant8({"q": x["q"], "s": x["s"]}, rows=False, cols=True, offsets=off)
    assert o["q"] is None and o["s"] is None
    v = _cols(_kept(x), off)
    _check_near(o["qc"], o["sc"], v, v.abs() * 2.0 ** -24, 128, 1, False)


# ---- products --------------------------------------------------------------

def _rand_codes(rows, cols, seed, spread=120.0):
    g = _gen(seed)
    return _padded((torch.randn(rows, cols, generator=g, device=DEV) * spread).clamp(-TOP, TOP).to(F8).float(), F8, 16)


def _rand_scales(seed, *shape):
    return torch.exp(torch.randn(*shape, generator=_gen(seed), device=DEV)) / 100


def _b(n):
    return -(-n // 128)


def _operands(M, N, K, E, grad, seed):
    depth = N if grad else K
    x = {"q": _rand_codes(M, depth, seed), "s": _rand_scales(seed + 1, _b(depth), M)}
    q = _rand_codes(max(E, 1) * N, K, seed + 2)
    w = {"q": q.view(E, N, K) if E else q, "s": _rand_scales(seed + 3, *((E,) if E else ()), _b(N), _b(K))}
    return x, w


def _w64(q, s):
    N, K = q.shape
    return q.to(F64) * s.to(F64).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _check_product(got, x, w, grad, off):
    xv = _kept(x)
    spans = [(0, 0, xv.shape[0])] if off is None else [(e, *off.tolist()[e:e + 2]) for e in range(len(off) - 1)]
    seen = torch.zeros(xv.shape[0], dtype=torch.bool, device=DEV)
    for e, a, b in spans:
        wv = _w64(w["q"], w["s"]) if off is None else _w64(w["q"][e], w["s"][e])
        wv = wv if grad else wv.t()
        ref, size = xv[a:b] @ wv, xv[a:b].abs() @ wv.abs()
        # a scale's product and the sum over the blocks add three operations each at most
        tol = HALF * ref.abs() + (wv.shape[0] + 3 * _b(wv.shape[0])) * U * size
        err = (got[a:b].to(F64) - ref).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
        seen[a:b] = True
    assert bool((got[~seen] == 0).all())


PRODUCTS = [(1, 1, 1), (1, 300, 2000), (3, 129, 17), (16, 512, 384), (17, 40, 130), (33, 256, 128), (64, 1000, 1000), (65, 128, 640), (127, 257, 255),
            (129, 384, 1024), (256, 256, 256), (257, 520, 136), (700, 1100, 900), (1000, 1462, 392)]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products(M, N, K, grad):
    x, w = _operands(M, N, K, 0, grad, M + N)
    y = (G.linear8_dx if grad else G.linear8)(x, w)
    assert y.dtype is BF and y.shape == (M, K if grad else N)
    _check_product(y, x, w, grad, None)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K", [(17, 256, 4096), (64, 257, 2049), (130, 2304, 1100), (200, 1024, 2304), (300, 128, 8192), (5, 5000, 136), (16, 2500, 1000), (9, 33, 4111)])
def test_products_of_few_rows(M, N, K, grad):
    """Sums cut into parts and joined, and up to sixteen tokens at every number of blocks."""
    x, w = _operands(M, N, K, 0, grad, M + N)
    _check_product((G.linear8_dx if grad else G.linear8)(x, w), x, w, grad, None)


EXPERTS = [(1, 64, 128, 4, 0, ()), (7, 136, 264, 64, 0, (0,)), (300, 256, 384, 3, 30, (1,)), (1000, 520, 200, 16, 100, (0, 7, 15)), (513, 128, 128, 2, 0, ()),
           (2000, 384, 256, 5, 0, (2,)), (40, 32, 32, 1024, 3, ()), (600, 128, 256, 300, 0, (5,)), (64, 128, 128, 3, 64, ())]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K,E,spare,empty", EXPERTS)
def test_products_by_expert(M, N, K, E, spare, empty, grad):
    x, w = _operands(M, N, K, E, grad, M + N)
    off = _offsets(M, E, M, spare, empty)
    _check_product((G.linear8_dx if grad else G.linear8)(x, w, offsets=off), x, w, grad, off)


def _check_dw(got, dy, x, off, E):
    C = dy["sc"].shape[0]
    dv, xv = ((o["qc"].to(F64).view(C, 128, -1) * o["sc"].to(F64)[:, None]) for o in (dy, x))
    half = HALF if got.dtype is BF else 2.0 ** -24
    spans = [(None, 0, C)] if off is None else [(e, a // 128 + e, a // 128 + e + _b(b - a)) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))]
    for e, b0, b1 in spans:
        d, v = dv[b0:b1].reshape(-1, dv.shape[2]), xv[b0:b1].reshape(-1, xv.shape[2])
        ref, size = d.t() @ v, d.abs().t() @ v.abs()
        tol = half * ref.abs() + 128 * (b1 - b0) * U * size + 4 * (b1 - b0) * U * size
        err = ((got if e is None else got[e]).to(F64) - ref).abs()
        assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_weight_gradients(M, N, K, dtype):
    dy, x = (G.quant8(_x(M, n, M + n), rows=False, cols=True) for n in (N, K))
    dw = G.linear8_dw(dy, x, dtype=dtype)
    assert dw.dtype is dtype and dw.shape == (N, K)
    _check_dw(dw, dy, x, None, 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K,E,spare,empty", [(4096, 256, 256, 0, 0, ()), (3000, 300, 513, 0, 0, ()), (2050, 17, 1000, 0, 0, ()),
                                                 (6000, 260, 200, 3, 100, (1,)), (5000, 128, 384, 2, 0, ())])
def test_weight_gradients_in_parts(M, N, K, E, spare, empty, dtype):
    """Long sums of few tiles, cut into parts (more of them than an expert has blocks) and joined."""
    off = _offsets(M, E, M, spare, empty) if E else None
    dy, x = (G.quant8(_x(M, n, M + n), rows=False, cols=True, offsets=off) for n in (N, K))
    _check_dw(G.linear8_dw(dy, x, offsets=off, dtype=dtype), dy, x, off, E)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K,E,spare,empty", EXPERTS)
def test_weight_gradients_by_expert(M, N, K, E, spare, empty, dtype):
    off = _offsets(M, E, M, spare, empty)
    dy, x = (G.quant8(_x(M, n, M + n), rows=False, cols=True, offsets=off) for n in (N, K))
    dw = G.linear8_dw(dy, x, offsets=off, dtype=dtype)
    assert dw.dtype is dtype and dw.shape == (E, N, K)
    _check_dw(dw, dy, x, off, E)


def test_every_code_multiplies_as_its_value():
    """All 254 finite codes on either side, one product each: exact in fp32, rounded once."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device=DEV)
    a = torch.zeros(254, 256, dtype=torch.uint8, device=DEV)
    a[:, 130] = codes
    w = {"q": a.view(F8), "s": torch.full((2, 2), 0.5, device=DEV)}
    x = {"q": a.view(F8), "s": torch.full((2, 254), 0.25, device=DEV)}
    v = codes.view(F8).to(F64)
    assert torch.equal(G.linear8(x, w), (v[:, None] * v[None, :] * 0.125).to(F32).to(BF))


def test_nan_scales_reach_their_rows_only():
    x, w = _operands(70, 300, 256, 0, False, 3)
    x["s"][1, 11] = float("nan")
    y = G.linear8(x, w)
    assert bool(torch.isnan(y[11]).all()) and int(torch.isnan(y).any(1).sum()) == 1
    # rows of the next expert share the tile's boxes; what they hold does not count
    x, w = _operands(300, 128, 256, 2, False, 4)
    off = torch.tensor([0, 150, 300], dtype=torch.int32, device=DEV)
    clean = G.linear8(x, w, offsets=off)
    x["q"].view(torch.uint8)[150:] = 0x7F
    again = G.linear8(x, w, offsets=off)
    assert torch.equal(again[:150], clean[:150]) and bool(torch.isnan(again[150:]).all())


# ---- the gated activation --------------------------------------------------

def _act64(act, x):
    if act == G.ACT_SILU:
        s, z = torch.sigmoid(x), torch.sigmoid(-x)
        return x * s, s + x * s * z
    if act == G.ACT_GELU_TANH:
        c = math.sqrt(2 / math.pi)
        t = 2 * c * (x + 0.044715 * x ** 3)
        s, z = torch.sigmoid(t), torch.sigmoid(-t)
        return x * s, s + x * s * z * 2 * c * (1 + 0.134145 * x * x)
    if act == G.ACT_RELU:
        return x.clamp_min(0), (x > 0).to(F64)
    if act == G.ACT_IDENTITY:
        return x, torch.ones_like(x)
    phi = 0.5 * torch.special.erfc(-x / math.sqrt(2))
    return x * phi, phi + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def _act_err(act, x):
    """Bounds of the kernels' errors for |x| up to 16, in units of the values' own
    arithmetic: (of act(x), of act'(x)).

    e^-t is computed from t = x or 2 c (x + 0.044715 x^3), whose rounding (five of
    2^-24 at most, one more for the product with log2 e) is |t| 2^-21 in the
    exponential, and 2^-21 for the functions.  s = 1 / (1 + e^-t) then has a
    relative error of (1 - s) r + 2^-22, r = (|t| + 1) 2^-21, and 1 - s an absolute
    one of s times that and 2^-24; where s is below 2^-126 it may be 0."""
    if act in (G.ACT_SILU, G.ACT_GELU_TANH):
        c = math.sqrt(2 / math.pi)
        t, k = (x, torch.ones_like(x)) if act == G.ACT_SILU else (2 * c * (x + 0.044715 * x ** 3), 2 * c * (1 + 0.134145 * x * x))
        s, z = torch.sigmoid(t), torch.sigmoid(-t)
        r = (t.abs() + 1) * 2.0 ** -21
        rs = z * r + 2.0 ** -21
        xk = x.abs() * k
        return x.abs() * (s * rs + 2.0 ** -126), s * ((1 + xk * z) * (rs + 2.0 ** -21) + xk * (s * rs + 2.0 ** -24)) + 2.0 ** -120
    if act == G.ACT_GELU_ERF:
        phi, pdf = 0.5 * torch.special.erfc(-x / math.sqrt(2)), torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        # CUDA's bound of normcdff, 5 units in the last place, and the products
        return x.abs() * (phi * 2.0 ** -20 + 2.0 ** -126), x.abs() * pdf * (x * x + 8) * 2.0 ** -22 + phi * 2.0 ** -20 + 2.0 ** -120
    return x.abs() * 0, x.abs() * 0


GLU = [(1, 1), (1, 1024), (5, 40), (64, 128), (65, 129), (130, 300), (33, 1462), (500, 256)]


def _gate(M, H, seed):
    """Gates up to 16: where the activations' errors are derived for."""
    return _padded(_x(M, H, seed, 2.0).float().clamp(-16, 16), BF)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,H", GLU)
def test_glu_forward(M, H, act):
    gate, up = _gate(M, H, M + H), _x(M, H, M + H + 1)
    o = G.glu8(gate, up, act=act)
    _check_exact(o["gate"]["q"], o["gate"]["s"], gate.to(F64), 1, 128, True)
    _check_exact(o["up"]["q"], o["up"]["s"], up.to(F64), 1, 128, True)
    g, u = gate.to(F64), up.to(F64)
    h = _act64(act, g)[0] * u
    err = _act_err(act, g)[0] * u.abs() + h.abs() * 2.0 ** -23
    _check_near(o["h"]["q"], o["h"]["s"], h, err, 1, 128, True)
    p = G.glu8(gate, up, act=act, h8=False)
    _same_bits(p["gate"]["q"], o["gate"]["q"])
    _same_bits(p["up"]["s"], o["up"]["s"])
    assert p["h"].dtype is BF and bool(((p["h"].to(F64) - h).abs() <= HALF * (h.abs() + err) + err + 2.0 ** -133).all())


def _kept_pair(M, H, seed):
    o = G.glu8(_gate(M, H, seed), _x(M, H, seed + 1), act=G.ACT_IDENTITY)
    return o["gate"], o["up"], _x(M, H, seed + 2, 0.1)


def _grads64(act, gate8, up8, dh):
    """(d, its error, h, its error); every product adds half a unit of fp32, and gate
    and up are rounded products themselves, which moves act by act' times that."""
    g, u, dy = _kept(gate8), _kept(up8), dh.to(F64)
    a, d = _act64(act, g)
    ea, ed = _act_err(act, g)
    ea = ea + g.abs() * 2.0 ** -23 * 1.2
    if act in (G.ACT_SILU, G.ACT_GELU_TANH, G.ACT_GELU_ERF):  # |act''| is below 1.2
        ed = ed + g.abs() * 2.0 ** -23 * 1.2
    d1, d2, h = dy * u * d, dy * a, a * u
    errors = torch.cat([(dy * u).abs() * (ed + d.abs() * 2.0 ** -21), dy.abs() * (ea + a.abs() * 2.0 ** -23)], 1)
    return torch.cat([d1, d2], 1), errors, h, u.abs() * (ea + a.abs() * 2.0 ** -22)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,H", GLU)
def test_glu_backward(M, H, act):
    gate8, up8, dh = _kept_pair(M, H, M + H)
    o = G.glu8_bwd(gate8, up8, dh, act=act)
    d, ed, h, eh = _grads64(act, gate8, up8, dh)
    assert o["d"].shape == (M, 2 * H) and o["h"].shape == (M, H)
    assert bool(((o["d"].to(F64) - d).abs() <= HALF * (d.abs() + ed) + ed + 2.0 ** -133).all())
    assert bool(((o["h"].to(F64) - h).abs() <= HALF * (h.abs() + eh) + eh + 2.0 ** -133).all())
    n = G.glu8_bwd(gate8, up8, dh, act=act, need_h=False)
    assert n["h"] is None and torch.equal(n["d"], o["d"])


@pytest.mark.parametrize("H", [*range(121, 138), 255, 257, 261])
def test_glu_backward_halves_at_every_offset(H):
    """dUp begins H elements behind a row's start: all remainders of eight, and what
    stands beside the matrices stays."""
    gate8, up8, dh = _kept_pair(19, H, H)
    wide = torch.full((19, -(-2 * H // 8) * 8 + 16), -7.0, dtype=BF, device=DEV)
    o = G.glu8_bwd(gate8, up8, dh, out={"d": wide[:, 8:8 + 2 * H]})
    d, ed, _, _ = _grads64(G.ACT_SILU, gate8, up8, dh)
    assert bool(((o["d"].to(F64) - d).abs() <= HALF * (d.abs() + ed) + ed + 2.0 ** -133).all())
    assert bool((wide[:, :8] == -7).all()) and bool((wide[:, 8 + 2 * H:] == -7).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,H,E,spare,empty", [(1, 128, 0, 0, ()), (200, 256, 0, 0, ()), (300, 128, 5, 40, (2,)), (1000, 384, 3, 0, ()), (20, 128, 64, 3, (0, 9))])
def test_glu_backward_quantised(M, H, E, spare, empty, act):
    gate8, up8, dh = _kept_pair(M, H, M + H)
    off = _offsets(M, E, M, spare, empty) if E else None
    o = G.glu8_bwd(gate8, up8, dh, act=act, quant=True, offsets=off)
    d, ed, h, eh = _grads64(act, gate8, up8, dh)
    _check_near(o["d"]["q"], o["d"]["s"], d, ed, 1, 128, True)
    _check_near(o["d"]["qc"], o["d"]["sc"], _cols(d, off), _cols(ed, off), 128, 1, False)
    _check_near(o["h"]["qc"], o["h"]["sc"], _cols(h, off), _cols(eh, off), 128, 1, False)
    n = G.glu8_bwd(gate8, up8, dh, act=act, quant=True, need_h=False, offsets=off)
    assert n["h"] is None
    for k in o["d"]:
        _same_bits(n["d"][k], o["d"][k])


@pytest.mark.parametrize("act", ACTS)
def test_glu_backward_against_differences(act):
    """dGate by central differences of the definition at the kept gate."""
    gate8, up8, dh = _kept_pair(40, 128, 77)
    o = G.glu8_bwd(gate8, up8, dh, act=act)
    g, u = _kept(gate8), _kept(up8)
    e = 1e-5
    diff = (_act64(act, g + e)[0] - _act64(act, g - e)[0]) / (2 * e)
    want = dh.to(F64) * u * diff
    keep = (g.abs() > 1e-3) if act == G.ACT_RELU else torch.ones_like(g, dtype=torch.bool)
    # third derivatives are below 3: e^2 / 2 of them, and the differences' own rounding 2^-52 |a| / e
    err = _grads64(act, gate8, up8, dh)[1][:, :128] + (dh.to(F64) * u).abs() * (3e-10 + 1e-10 * g.abs())
    tol = HALF * (want.abs() + err) + err
    assert bool(((o["d"][:, :128].to(F64) - want).abs() <= tol)[keep].all())


@pytest.mark.parametrize("act", ACTS)
def test_glu_of_large_gates(act):
    """Far out act is 0 or z and act' 0 or 1, up to bf16's largest values."""
    top = float(torch.finfo(BF).max)
    g = torch.tensor([1e4, -1e4, 1e19, -1e19, 1e30, -1e30, top, -top] * 16, device=DEV, dtype=BF).repeat(16, 1).t().contiguous()
    up = torch.full((128, 16), 2.0 ** -120, dtype=BF, device=DEV)
    o = G.glu8(g, up, act=act, h8=False)
    z = g.to(F64)
    a = z if act == G.ACT_IDENTITY else z.clamp_min(0)
    want = a * 2.0 ** -120
    assert bool(((o["h"].to(F64) - want).abs() <= HALF * want.abs()).all())
    b = G.glu8_bwd(o["gate"], o["up"], torch.ones(128, 16, dtype=BF, device=DEV), act=act)
    d = torch.ones_like(z) if act == G.ACT_IDENTITY else (z > 0).to(F64)
    u, k = _kept(o["up"]), _kept(o["gate"])
    assert bool(((b["d"][:, :16].to(F64) - u * d).abs() <= HALF * u).all())
    a = k if act == G.ACT_IDENTITY else k.clamp_min(0)
    assert bool(((b["d"][:, 16:].to(F64) - a).abs() <= HALF * a.abs()).all())


def test_glu_nan_stays_in_its_block():
    gate, up = _x(40, 256, 1), _x(40, 256, 2)
    gate[5, 3], up[9, 200] = float("nan"), float("inf")
    o = G.glu8(gate, up)
    for key, row, block in (("gate", 5, 0), ("up", 9, 1), ("h", 5, 0), ("h", 9, 1)):
        bad = torch.isnan(o[key]["s"])
        assert bool(bad[block, row]) and int(bad.sum()) == (2 if key == "h" else 1)
    b = G.glu8_bwd(o["gate"], o["up"], _x(40, 256, 3), quant=True)
    bad = torch.isnan(b["d"]["s"])
    assert bool(bad[0, 5]) and bool(bad[2, 5]) and bool(bad[1, 9]) and not bool(bad[3, 9]) and int(bad.sum()) == 3
    assert int(torch.isnan(b["d"]["sc"]).sum()) == 128 * 3 and int(torch.isnan(b["h"]["sc"]).sum()) == 256


def test_codes_of_products_of_bf16_are_exact():
    """h without a rounding ahead of its own (ReLU, identity): products of two bf16 are
    exact in fp32, so their codes and scales are the definition's, midpoints included."""
    for act in (G.ACT_RELU, G.ACT_IDENTITY):
        for H, cut in ((2048, 0xFFFF0000), (2048, 0xFFE00000), (1000, 0xFFFF0000)):  # full mantissas; three bits, where midpoints abound
            gate, up = ((_x(1000, H, H + s).float().view(torch.int32) & (cut - (1 << 32))).view(F32) for s in (0, 1))
            gate, up = _padded(gate, BF), _padded(up, BF)
            h = _act64(act, gate.to(F64))[0] * up.to(F64)
            o = G.glu8(gate, up, act=act)
            _check_exact(o["h"]["q"], o["h"]["s"], h, 1, 128, True)


def test_kept_rows_with_scales_of_powers_of_two():
    """Then the kept values are exact in fp32, quotients are midpoints or 2^-9 away from
    one, and 448 / a rounded once decides all of them: the definition's codes."""
    q = _rand_codes(1000, 512, 3)
    s = _power(torch.randint(-9, 9, (4, 1000), generator=_gen(4), device=DEV)).to(F32)
    x = {"q": q, "s": s}
    o = G.quant8(x, rows=False, cols=True)
    v = _cols(_kept(x), None)
    _check_exact(o["qc"], o["sc"], v, 128, 1, False)
    t = (v * TOP / _tile(v, 128, 1)[0]).abs()
    half = _power((torch.frexp(t)[1] - 1).clamp_min(-6) - 4)
    assert int(((t / half) % 2 == 1).sum()) > 1000  # there were midpoints


def test_kept_codes_are_within_four_roundings():
    """A kept value, its block's maximum, 448 / maximum and their product are rounded to
    fp32 once each, 2^-24 of them at most, and nothing else comes before the code.  How
    many codes differ from the definition's says nothing here: rows of bf16 often share a
    scale s, their values c s are rounded one by one, and a quotient c / c' of two codes
    of 4 bits that is a midpoint is then passed to either side."""
    x = G.quant8(_x(4096, 4096, 8))
    o = G.quant8({"q": x["q"], "s": x["s"]}, rows=False, cols=True)
    v = _cols(_kept(x), None)
    t = v * TOP / _tile(v, 128, 1)[0]
    d = t.abs() * (4 * 2.0 ** -24 + 2.0 ** -45)
    q = o["qc"].to(F64)
    assert bool(((q >= _e4m3(t - d)) & (q <= _e4m3(t + d))).all())


def test_kept_quotients_next_to_borders():
    """Codes of 1 stand for their scales, any fp32: 448 / maximum and its product with the
    value are then the only roundings, 2^-23 of a quotient together.  Values whose
    quotients are that and a little more from a border between two codes get the
    definition's code."""
    blocks, M = 1024, 256
    g = _gen(12)
    a = torch.exp(2 * torch.randn(1, blocks, generator=g, device=DEV)).to(F64)
    odd = 2 * torch.randint(8, 16, (M, blocks), generator=g, device=DEV) + 1
    q = odd.to(F64) * _power(torch.randint(-6, 4, (M, blocks), generator=g, device=DEV))  # up to 31 * 8, below 448
    v = (q * a / TOP).to(F32)
    v = (v.view(torch.int32) + torch.randint(-3, 4, (M, blocks), generator=g, device=DEV, dtype=torch.int32)).view(F32)
    v[::128] = a.to(F32)
    x = {"q": torch.ones(M, 128 * blocks, dtype=F8, device=DEV), "s": v.t().contiguous()}
    o = G.quant8(x, rows=False, cols=True)
    a = a.to(F32).to(F64)
    t = v.to(F64) * TOP / a
    away = (t - q).abs() > q * (2.0 ** -23 + 2.0 ** -40)
    away[::128] = False  # the maxima themselves
    got = o["qc"].view(M, blocks, 128).to(F64)
    assert bool((got == got[:, :, :1]).all()) and bool((got[::128] == TOP).all())
    assert int(away.sum()) > M * blocks // 4
    assert torch.equal(got[:, :, 0][away], _e4m3(t)[away])


def test_zeros_among_other_values_keep_their_sign():
    x = _x(130, 256, 21)
    x[:, ::3], x[:, 1::3] = -0.0, 0.0
    o = G.quant8(x, rows=True, cols=True)
    for q in (o["q"], o["qc"][:130], G.quant8_weight(x)["q"], G.glu8(x, x)["gate"]["q"]):
        assert bool((q[:, ::3].view(torch.uint8) == 0x80).all()) and bool((q[:, 1::3].view(torch.uint8) == 0).all())


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 2048, 2048), (1, 4096, 4096), (1, 2049, 1000), (1, 1000, 2049), (1, 8192, 7168), (2, 8192, 7168)])
def test_products_of_one_and_two_deep_rows(M, N, K, grad):
    """One token's sum is cut into parts too, where the gradient's is deep."""
    x, w = _operands(M, N, K, 0, grad, M + N)
    _check_product((G.linear8_dx if grad else G.linear8)(x, w), x, w, grad, None)


@pytest.mark.parametrize("M,N,K,E", [(300, 130, 200, 0), (2000, 256, 136, 0), (700, 128, 260, 3)])
def test_weight_gradients_sum_in_all_of_fp32(M, N, K, E):
    """Whole numbers whose sums stay below 2^24 are summed exactly where every addition
    keeps 24 bits: large products next to ones, and scales of powers of two that move
    whole blocks up and down.  A sum that keeps fewer bits anywhere loses the ones."""
    off = _offsets(M, E, M, 20) if E else None
    C = M // 128 + E if E else _b(M)
    g = _gen(M)

    def codes(n):
        big = torch.rand(128 * C, n, generator=g, device=DEV) < 0.02
        v = torch.where(big, TOP, 1.0) * (1 - 2 * torch.randint(0, 2, (128 * C, n), generator=g, device=DEV))
        return _padded(v.to(F8).float(), F8, 16)
    s = [2.0 ** torch.randint(-1, 2, (C, 1), generator=g, device=DEV) for _ in range(2)]  # products are multiples of 1 / 4
    dy, x = ({"qc": codes(n), "sc": c.expand(C, n).contiguous()} for n, c in zip((N, K), s))
    dv, xv = (o["qc"].to(F64) * o["sc"].to(F64).repeat_interleave(128, 0) for o in (dy, x))
    dw = G.linear8_dw(dy, x, offsets=off, dtype=F32)
    spans = [(None, 0, C)] if off is None else [(e, a // 128 + e, a // 128 + e + _b(b - a)) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))]
    for e, b0, b1 in spans:
        d, v = dv[128 * b0:128 * b1], xv[128 * b0:128 * b1]
        assert d.numel() == 0 or float((d.abs().t() @ v.abs()).max()) * 4 < 2.0 ** 24  # any order of them is exact
        assert torch.equal((dw if e is None else dw[e]).to(F64), d.t() @ v)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(1, 130, 2000, 0), (16, 2000, 300, 0), (40, 2048, 2048, 0), (300, 260, 1000, 0), (200, 256, 384, 3), (700, 128, 512, 2)])
def test_products_sum_in_all_of_fp32(M, N, K, E, grad):
    """The same of y and dx: exact sums below 2^24, rounded to bf16 once."""
    depth, width = (N, K) if grad else (K, N)
    g = _gen(M)

    def codes(rows, n):
        big = torch.rand(rows, n, generator=g, device=DEV) < 0.02
        v = torch.where(big, TOP, 1.0) * (1 - 2 * torch.randint(0, 2, (rows, n), generator=g, device=DEV))
        return _padded(v.to(F8).float(), F8, 16)
    q = codes(max(E, 1) * N, K)
    w = {"q": q.view(E, N, K) if E else q, "s": 2.0 ** torch.randint(-1, 2, (*((E,) if E else ()), _b(N), _b(K)), generator=g, device=DEV)}
    x = {"q": codes(M, depth), "s": 2.0 ** torch.randint(-1, 2, (_b(depth), M), generator=g, device=DEV)}
    off = _offsets(M, E, M, 7) if E else None
    y = (G.linear8_dx if grad else G.linear8)(x, w, offsets=off)
    xv = _kept(x)
    for e, a, b in [(None, 0, M)] if off is None else [(e, *off.tolist()[e:e + 2]) for e in range(E)]:
        wv = _w64(w["q"], w["s"]) if e is None else _w64(w["q"][e], w["s"][e])
        wv = wv if grad else wv.t()
        assert a == b or float((xv[a:b].abs() @ wv.abs()).max()) * 4 < 2.0 ** 24
        assert torch.equal(y[a:b], (xv[a:b] @ wv).to(F32).to(BF))
