"""The operators in 8 bits together, as the example runs them, and the ways in which a
program may call them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import expert_ffn8 as X  # noqa: E402
import fp4_quant_gb300 as G  # noqa: E402

DEV = torch.device("cuda:0")
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _rand(*shape, seed, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)).to(BF)


def _sorted(R, E, seed):
    ids = torch.randint(-1, E, (R, 1), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    return G.route(ids, E)


def _reference(xs, w, offsets, dy):
    t = {k: v.double().requires_grad_(True) for k, v in {**w, "xs": xs}.items()}
    H = w["down"].shape[2]
    cuts = offsets.tolist()
    rows = [torch.zeros(0, xs.shape[1], dtype=torch.float64, device=DEV)]
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        u = t["xs"][a:b] @ t["up"][e].t()
        rows.append((torch.nn.functional.silu(u[:, :H]) * u[:, H:]) @ t["down"][e].t())
    y = torch.cat(rows)
    (y * dy[:cuts[-1]].double()).sum().backward()
    return y.detach(), {k: v.grad for k, v in t.items()}


@pytest.mark.parametrize("R,D,H,E", [(1, 128, 128, 4), (100, 264, 128, 6), (700, 512, 256, 16), (1500, 256, 384, 3)])
def test_experts_forward_and_backward(R, D, H, E):
    w = X.make_weights(D, H, E, seed=R)
    xs, dy = _rand(R, D, seed=R + 1), _rand(R, D, seed=R + 2)
    off = _sorted(R, E, R + 3)["offsets"]
    used = int(off[-1])
    w8 = X.quantise(w)
    y, s = X.forward(xs, w8, off)
    g = X.backward(dy, w8, s, off)
    want_y, want = _reference(xs, w, off, dy)
    # roundings to E4M3 one behind the other: x, up, h, down in y; x or dy, down, dh's
    # operands, gate, up, d and the other operand in the gradients: seven at most, 2^-4
    # each at worst relative to the norm of what they round
    assert bool((y[used:] == 0).all()) and bool((g["xs"][used:] == 0).all())
    for name, a, b in [("y", y[:used], want_y)] + [(n, g[n], want[n]) for n in g]:
        assert a.shape == b.shape and float((a.double() - b).norm()) <= 7 * 2.0 ** -4 * float(b.norm()), name
    empty = [e for e in range(E) if int(off[e]) == int(off[e + 1])]
    assert all(bool((g[n][empty] == 0).all()) for n in ("up", "down"))


def _calls(seed):
    """Every call once, small; what they return, flat."""
    off = torch.tensor([0, 40, 40, 190, 200], dtype=torch.int32, device=DEV)
    x, dy = _rand(210, 256, seed=seed), _rand(210, 128, seed=seed + 1)
    w = G.quant8_weight(_rand(4, 128, 256, seed=seed + 2, scale=0.1))
    gate, up, dh = (_rand(210, 256, seed=seed + 3 + i) for i in range(3))
    deep, deep_w = G.quant8(_rand(64, 4096, seed=seed + 6)), G.quant8_weight(_rand(264, 4096, seed=seed + 7, scale=0.1))  # a sum in parts

    def run():
        x8 = G.quant8(x, cols=True, offsets=off)
        d8 = G.quant8(dy, cols=True, offsets=off)
        a = G.glu8(gate, up)
        b = G.glu8_bwd(a["gate"], a["up"], dh, quant=True, offsets=off)
        p = G.glu8_bwd(a["gate"], a["up"], dh)
        k = G.quant8({"q": x8["q"], "s": x8["s"]}, rows=False, cols=True, offsets=off)
        few = {"q": x8["q"][:1], "s": x8["s"][:, :1].contiguous()}
        one = {"q": w["q"][0], "s": w["s"][0]}
        return [x8["q"], x8["s"], x8["qc"], x8["sc"], k["qc"], k["sc"], G.linear8(x8, w, offsets=off), G.linear8_dx(d8, w, offsets=off),
                G.linear8_dw(d8, x8, offsets=off), G.linear8_dw(d8, x8, offsets=off, dtype=torch.float32), G.linear8(few, one), G.linear8(x8, one), G.linear8(deep, deep_w),
                a["h"]["q"], a["h"]["s"], a["gate"]["q"], a["up"]["s"], *b["d"].values(), *b["h"].values(), p["d"], p["h"],
                w["q"], w["s"]]
    return run


def _equal(a, b):
    return all(torch.equal(p.view(torch.uint8) if p.dtype is F8 else p, q.view(torch.uint8) if q.dtype is F8 else q) for p, q in zip(a, b))


def test_calls_repeat_bit_for_bit():
    run = _calls(1)
    first = run()
    assert all(_equal(first, run()) for _ in range(3))


def test_calls_in_a_graph_and_two_graphs_at_once():
    runs = [_calls(10), _calls(20)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for o in outs:
            for t in o[:-2]:  # the last two are the weights, quantised outside the graphs: their inputs
                t.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(_equal(a[:-2], b[:-2]) for a, b in zip(outs, want))


def test_calls_on_a_given_stream():
    x = _rand(300, 384, seed=5)
    w = _rand(256, 384, seed=6, scale=0.1)
    want = G.linear8(G.quant8(x), G.quant8_weight(w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        y = G.linear8(G.quant8(x, stream=stream), G.quant8_weight(w, stream=stream), stream=stream)
        s.synchronize()
        assert torch.equal(y, want)


def test_outputs_given_and_what_stands_beside_them():
    x, w = _rand(70, 136, seed=7), _rand(200, 136, seed=8)
    x8, w8 = G.quant8(x, cols=True), G.quant8_weight(w)
    q = torch.full((70, 176), 7, dtype=torch.uint8, device=DEV)
    qc = torch.full((128, 160), 7, dtype=torch.uint8, device=DEV)
    o = G.quant8(x, cols=True, out={"q": q[:, :136].view(F8), "qc": qc[:, 16:152].view(F8)})
    assert _equal([o["q"], o["qc"], o["s"], o["sc"]], [x8["q"], x8["qc"], x8["s"], x8["sc"]])
    assert bool((q[:, 136:] == 7).all()) and bool((qc[:, :16] == 7).all()) and bool((qc[:, 152:] == 7).all())
    y = torch.full((70, 208), -7.0, dtype=BF, device=DEV)
    G.linear8(x8, w8, out=y[:, :200])
    assert torch.equal(y[:, :200], G.linear8(x8, w8)) and bool((y[:, 200:] == -7).all())
    d8 = G.quant8(_rand(70, 200, seed=9), rows=False, cols=True)
    dw = torch.full((200, 144), -7.0, device=DEV)
    G.linear8_dw(d8, x8, dtype=torch.float32, out=dw[:, :136])
    assert torch.equal(dw[:, :136], G.linear8_dw(d8, x8, dtype=torch.float32)) and bool((dw[:, 136:] == -7).all())
    a = G.glu8(x, x)
    d = torch.full((70, 280), -7.0, dtype=BF, device=DEV)
    b = G.glu8_bwd(a["gate"], a["up"], x, out={"d": d[:, :272]})
    assert b["d"].data_ptr() == d.data_ptr() and bool((d[:, 272:] == -7).all())
    assert torch.equal(d[:, :272], G.glu8_bwd(a["gate"], a["up"], x)["d"])


def test_column_forms_of_parts_and_views():
    """Halves of a projection, slices of a wider matrix: strides of their own."""
    wide = _rand(150, 512, seed=11)
    for view in (wide[:, 128:384], wide[:, 256:], wide[20:]):
        a, b = G.quant8(view, cols=True), G.quant8(view.contiguous(), cols=True)
        assert _equal([v for v in a.values()], [v for v in b.values()])
    a, b = G.glu8(wide[:, :256], wide[:, 256:]), G.glu8(wide[:, :256].contiguous(), wide[:, 256:].contiguous())
    assert _equal([a[k][n] for k in a for n in ("q", "s")], [b[k][n] for k in b for n in ("q", "s")])
    odd = _rand(33, 67, seed=12)  # contiguous rows that do not start on 16 bytes are copied first
    padded = torch.zeros(33, 72, dtype=BF, device=DEV)
    padded[:, :67] = odd
    assert _equal(list(G.quant8(odd, cols=True).values()), list(G.quant8(padded[:, :67], cols=True).values()))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    M, K = (1 << 18) + 5, 8200
    x = torch.empty(M, K, dtype=BF, device=DEV).fill_(0.5)
    x[-300:] = _rand(300, K, seed=1)
    big, last = G.quant8(x, cols=True), G.quant8(x[-133:], cols=True)  # 133 = 128 + M % 128: the last two column blocks
    assert _equal([big["q"][-133:], big["s"][:, -133:], big["qc"][-256:], big["sc"][-2:]], [last["q"], last["s"], last["qc"], last["sc"]])
    again = G.quant8({"q": big["q"], "s": big["s"]}, rows=False, cols=True)
    assert _equal([again["qc"][-256:]], [G.quant8({"q": last["q"], "s": last["s"]}, rows=False, cols=True)["qc"]])
    del again, last
    a, b = G.glu8(x, x), G.glu8(x[-133:], x[-133:])
    assert _equal([a["h"]["q"][-133:], a["gate"]["s"][:, -133:]], [b["h"]["q"], b["gate"]["s"]])
    d = G.glu8_bwd(a["gate"], a["up"], x)
    assert torch.equal(d["d"][-133:], G.glu8_bwd(b["gate"], b["up"], x[-133:])["d"])


def test_products_with_results_beyond_32_bits():
    M, N, K = 1 << 17, 16520, 128
    x8 = G.quant8(_rand(M, K, seed=2))
    w8 = G.quant8_weight(_rand(N, K, seed=3))
    y = G.linear8(x8, w8)
    tail = {"q": x8["q"][-300:], "s": x8["s"][:, -300:].contiguous()}
    assert torch.equal(y[-300:], G.linear8(tail, w8)) and torch.equal(y[:20], G.linear8({"q": x8["q"][:20], "s": x8["s"][:, :20].contiguous()}, w8))
    del y
    E, N, K = 64, 8192, 4104
    off = torch.tensor([0] * (E - 1) + [100, 300], dtype=torch.int32, device=DEV)
    d8, x8 = (G.quant8(_rand(300, n, seed=n), rows=False, cols=True, offsets=off) for n in (N, K))
    dw = G.linear8_dw(d8, x8, offsets=off)
    b = 100 // 128 + E - 1  # the last expert's two blocks
    alone = G.linear8_dw(*({"qc": t["qc"][128 * b:128 * b + 256], "sc": t["sc"][b:b + 2].contiguous()} for t in (d8, x8)))
    assert torch.equal(dw[-1], alone) and bool((dw[1:E - 2] == 0).all())


def test_calls_on_two_streams_at_once():
    x, w, dy = _rand(600, 1024, seed=20), G.quant8_weight(_rand(1024, 1024, seed=21, scale=0.1)), _rand(600, 1024, seed=22)
    x8, d8 = G.quant8(x, cols=True), G.quant8(dy, cols=True)
    few = {"q": x8["q"][:9], "s": x8["s"][:, :9].contiguous()}
    want = [G.linear8(x8, w), G.linear8_dx(d8, w), G.linear8_dw(d8, x8), G.linear8(few, w), G.glu8(x, dy)["h"]["q"]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(5):
        for s in streams:
            got.append([G.linear8(x8, w, stream=s), G.linear8_dx(d8, w, stream=s), G.linear8_dw(d8, x8, stream=s), G.linear8(few, w, stream=s),
                        G.glu8(x, dy, stream=s)["h"]["q"]])
    torch.cuda.synchronize()
    assert all(_equal(g, want) for g in got)


def test_offsets_out_of_range_stay_inside():
    """Cuts past the last row count as the last row; nothing outside is touched."""
    x, w = _rand(200, 256, seed=30), G.quant8_weight(_rand(3, 128, 256, seed=31))
    good = torch.tensor([0, 50, 200, 200], dtype=torch.int32, device=DEV)
    wild = torch.tensor([0, 50, 10 ** 6, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    a, b = G.quant8(x, cols=True, offsets=good), G.quant8(x, cols=True, offsets=wild)
    assert _equal([a["q"], a["qc"], a["sc"]], [b["q"], b["qc"], b["sc"]])
    assert torch.equal(G.linear8(a, w, offsets=good), G.linear8(a, w, offsets=wild))
    for bad in ([0, -5, 70, 200], [0, 150, 20, 300], [7, 3, 2, 1], [2 ** 31 - 1, 0, -1, 5]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        q = G.quant8(x, cols=True, offsets=off)
        G.linear8(a, w, offsets=off)
        G.linear8_dx(G.quant8(_rand(200, 128, seed=32)), w, offsets=off)
        G.linear8_dw(q, q, offsets=off)
        g = G.glu8(x, x)
        G.glu8_bwd(g["gate"], g["up"], x, quant=True, offsets=off)
    torch.cuda.synchronize()
    assert torch.equal(G.linear8(a, w, offsets=good), G.linear8(a, w, offsets=wild))


def test_one_expert_of_a_stack():
    """Matrices and scales out of a stack's, whose scales begin at any word."""
    w = G.quant8_weight(_rand(3, 300, 136, seed=40))  # 3 x 2 scales each
    x = G.quant8(_rand(1, 136, seed=41))
    many = G.quant8(_rand(151, 136, seed=42), cols=True)
    for e in range(3):
        one = {"q": w["q"][e], "s": w["s"][e]}
        q = torch.zeros(300, 144, dtype=torch.uint8, device=DEV)[:, :136]
        own = {"q": q.copy_(w["q"][e].view(torch.uint8)).view(F8), "s": w["s"][e].clone()}
        assert torch.equal(G.linear8(x, one), G.linear8(x, own)) and torch.equal(G.linear8(many, one), G.linear8(many, own))
    # one block of a row form's columns, one block of a column form's rows
    part = {"q": many["q"][:, 128:], "s": many["s"][1:]}
    whole = torch.zeros(151, 16, dtype=torch.uint8, device=DEV)[:, :8].copy_(part["q"].view(torch.uint8))
    a, b = G.quant8(part, rows=False, cols=True), G.quant8({"q": whole.view(F8), "s": many["s"][1:].clone()}, rows=False, cols=True)
    assert _equal([a["qc"], a["sc"]], [b["qc"], b["sc"]])
    d = {"qc": many["qc"][128:], "sc": many["sc"][1:]}
    own = {"qc": d["qc"], "sc": d["sc"].clone()}
    assert torch.equal(G.linear8_dw(d, d), G.linear8_dw(own, own))


@pytest.mark.parametrize("R,D,H", [(1, 128, 67), (40, 136, 67), (129, 264, 130), (33, 128, 1462), (20, 64, 1)])
def test_halves_of_a_projection_of_any_width(R, D, H):
    """The second half of a projection begins on 16 bytes only where its width is a
    multiple of eight: forward and backward take it as they take an aligned copy."""
    x8, w8 = G.quant8(_rand(R, D, seed=H)), G.quant8_weight(_rand(2 * H, D, seed=H + 1, scale=0.1))
    u = G.linear8(x8, w8)
    dh = G.linear8(x8, w8)[:, H:]

    def aligned(t):
        buf = torch.zeros(t.shape[0], -(-t.shape[1] // 8) * 8, dtype=BF, device=DEV)[:, :t.shape[1]]
        return buf.copy_(t)
    a, b = G.glu8(u[:, :H], u[:, H:]), G.glu8(aligned(u[:, :H]), aligned(u[:, H:]))
    assert _equal([a[k][n] for k in a for n in ("q", "s")], [b[k][n] for k in b for n in ("q", "s")])
    c, d = G.glu8_bwd(a["gate"], a["up"], dh), G.glu8_bwd(b["gate"], b["up"], aligned(dh))
    assert torch.equal(c["d"], d["d"]) and torch.equal(c["h"], d["h"])
    assert _equal(list(G.quant8(u[:, H:], cols=True).values()), list(G.quant8(aligned(u[:, H:]), cols=True).values()))


def _beside(rows, cols, dtype=F8, left=16):
    """A matrix inside a wider one of sevens, and a check that nothing but it was written."""
    ld = left + -(-cols // 16) * 16 + 16
    buf = torch.full((rows + 2, ld * dtype.itemsize), 7, dtype=torch.uint8, device=DEV)
    t = buf.view(dtype)[1:-1, left:left + cols]

    def kept():
        b = buf.clone()
        b.view(dtype)[1:-1, left:left + cols].view(torch.uint8).fill_(7)
        return bool((b == 7).all())
    return t, kept


@pytest.mark.parametrize("M,H,E", [(70, 128, 0), (70, 256, 3), (300, 384, 5)])
def test_every_output_may_be_given(M, H, E):
    """Outputs inside wider matrices are those of calls that allocate them, and what
    stands around them is left alone."""
    x, up, dh = (_rand(M, H, seed=M + i) for i in range(3))
    off = torch.tensor([round(M * e / E * 0.9) for e in range(E + 1)], dtype=torch.int32, device=DEV) if E else None
    C = M // 128 + E if E else -(-M // 128)
    checks = []

    def codes(rows, cols):
        t, kept = _beside(rows, cols)
        checks.append(kept)
        return t
    rows = lambda n: {"q": codes(M, n), "s": torch.empty(-(-n // 128), M, device=DEV)}  # noqa: E731
    cols = lambda n: {"qc": codes(128 * C, n), "sc": torch.empty(C, n, device=DEV)}  # noqa: E731

    def same(a, b):
        for k in b:
            if isinstance(b[k], dict):
                same(a[k], b[k])
            elif b[k] is not None:
                assert _equal([a[k]], [b[k]]), k
    both = {**rows(H), **cols(H)}
    x8 = G.quant8(x, cols=True, offsets=off, out=both)
    assert x8["qc"].data_ptr() == both["qc"].data_ptr()
    same(x8, G.quant8(x, cols=True, offsets=off))
    one = {"q": x8["q"].clone(memory_format=torch.contiguous_format), "s": x8["s"]}
    same(G.quant8(one, rows=False, cols=True, offsets=off, out=cols(H)), G.quant8(one, rows=False, cols=True, offsets=off))
    given = {"h": rows(H), "gate": rows(H), "up": rows(H)}
    a = G.glu8(x, up, out=given)
    same(a, G.glu8(x, up))
    h, kept = _beside(M, H, BF)
    checks.append(kept)
    same(G.glu8(x, up, h8=False, out={"h": h, "gate": given["gate"]}), G.glu8(x, up, h8=False))
    d = {**rows(2 * H), **cols(2 * H)}
    same(G.glu8_bwd(a["gate"], a["up"], dh, quant=True, offsets=off, out={"d": d, "h": cols(H)}),
         G.glu8_bwd(a["gate"], a["up"], dh, quant=True, offsets=off))
    w = _rand(max(E, 1), 136, H, seed=9)
    w = w if E else w[0]
    big = torch.full((max(E, 1), 136 + 3, H + 32), 7, dtype=torch.uint8, device=DEV)
    q = big[:, 1:-2, 16:16 + H].view(F8)
    w8 = G.quant8_weight(w, out={"q": q if E else q[0]})
    same(w8, G.quant8_weight(w))
    for o, call in ((_beside(M, 136, BF), lambda out: G.linear8(x8, w8, offsets=off, out=out)),
                    (_beside(M, H, BF), lambda out: G.linear8_dx(G.quant8(_rand(M, 136, seed=3)), w8, offsets=off, out=out))):
        checks.append(o[1])
        assert torch.equal(call(o[0]), call(None))
    big[:, 1:-2, 16:16 + H] = 7
    assert bool((big == 7).all()) and all(k() for k in checks)


def test_a_captured_layer_reads_its_inputs_at_every_replay():
    R, D, H, E = 600, 264, 256, 5
    w8 = X.quantise(X.make_weights(D, H, E, seed=1))
    off = _sorted(R, E, 2)["offsets"]
    xs, dy = _rand(R, D, seed=3), _rand(R, D, seed=4)

    def step():
        y, s = X.forward(xs, w8, off)
        return [y, *X.backward(dy, w8, s, off).values()]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (5, 6):
        xs.copy_(_rand(R, D, seed=seed))
        dy.copy_(_rand(R, D, seed=seed + 10))
        off.copy_(_sorted(R, E, seed + 20)["offsets"])
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert _equal(kept, step())
