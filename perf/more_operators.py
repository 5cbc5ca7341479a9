"""Timed cases of the operators in 8-bit floating point with a scale for each block of 128.

Each case is one call that a program makes:

* ``quant8``, ``quant8_weight``: a matrix as E4M3 codes with an fp32 scale per 1 x 128 (rows), 128 x 1 (columns) or
  128 x 128 (weights) block; ``again``: the column form made from the row form that a forward pass kept;
* ``linear8``, ``linear8_dx``, ``linear8_dw``: the matrix products of such operands, dense or by expert;
* ``glu8``, ``glu8_bwd``: the gated activation that keeps gate and up in 8 bits, and its backward from those.

A block's scale is a / 448 with a its largest absolute value (2^-100 at least), its codes are value * 448 / a rounded
to E4M3.  By expert the column blocks of expert e begin at block ``offsets[e] // 128 + e``, and its last one ends in
zeros; blocks that no expert has are zeros.

``run`` computes it in elementary torch operations in fp32, rounded once at the end (``own`` false), or by the
package's calls (``own`` true).  ``exact`` restates the definitions in fp64.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 128
TOP = 448.0
LEAST = 2.0 ** -100
ACTS = {"silu": 0, "gelu_tanh": 1, "relu": 2, "identity": 3, "gelu_erf": 4}  # the package's ACT_* values
F8, BF, F32, F64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.float64


# ---- cases ----------------------------------------------------------------

def _quant(M, K, mode, E=0, spare=0.0):
    return dict(op="quant", M=M, K=K, mode=mode, E=E, spare=spare)


def _product(kind, M, N, K, E=0, spare=0.0, wide=False):
    return dict(op="product", kind=kind, M=M, N=N, K=K, E=E, spare=spare, wide=wide)


def _glu(kind, M, H, act, E=0, spare=0.0):
    return dict(op="glu", kind=kind, M=M, H=H, act=act, E=E, spare=spare)


def listed():
    return [
        # the input of one token's projection in a decoding step
        dict(_quant(1, 8192, "rows"), name="quant_one_token"),
        # the gradient of a training batch, as the operand of both products of a backward pass
        dict(_quant(4096, 7168, "both"), name="quant_grad"),
        # the gate/up weights of 64 experts after an optimiser step
        dict(_quant(2048, 2048, "weights", E=64), name="quant_weights"),
        # the input that the experts' forward pass kept in 8 bits, for their weight gradients
        dict(_quant(32768, 2048, "again", E=64), name="quant_kept_input"),
        # one token's down projection: reading the weights is all there is
        dict(_product("fwd", 1, 7168, 8192), name="product_one_token"),
        # up projection of a training batch
        dict(_product("fwd", 4096, 8192, 7168), name="product_train"),
        # its input gradient, ragged token count
        dict(_product("dx", 4095, 8192, 7168), name="product_dx"),
        # the experts' gate/up projection: 32768 routed rows over 64 experts
        dict(_product("fwd", 32768, 2048, 2048, E=64), name="product_experts"),
        # its weight gradients
        dict(_product("dw", 32768, 2048, 2048, E=64), name="product_dw_experts"),
        # gated activation of a training batch: operand of the down projection, gate and up kept in 8 bits
        dict(_glu("fwd", 4096, 7168, "silu"), name="glu_train"),
        # backward from the kept gate and up, in bf16; ragged sizes
        dict(_glu("bwd", 8191, 1462, "gelu_tanh"), name="glu_bwd_ragged"),
        # the experts' backward, straight to the operands of the four products that follow
        dict(_glu("bwd8", 32768, 1024, "silu", E=64), name="glu_bwd_experts"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "glu"])
    E = rng.choice([0, 4, 8, 32, 64])
    spare = rng.choice([0.0, 0.05]) if E else 0.0
    if op == "quant":
        mode = rng.choice(["rows", "both", "weights", "again"])
        K = _log(rng, 256, 8192)
        K = K // 128 * 128 if rng.random() < 0.5 else K
        if mode == "weights":
            M = _log(rng, 256, 4096)
            return _quant(min(M, (1 << 28) // (K * max(E, 1))), K, mode, E)
        if mode == "rows":
            E, spare = 0, 0.0
        return _quant(min(_log(rng, 1, 32768), (1 << 26) // K), K, mode, E, spare)
    if op == "product":
        kind = rng.choice(["fwd", "dx", "dw"])
        if E:
            N, K, M = _log(rng, 256, 2048), _log(rng, 256, 2048), _log(rng, 8, 32768)
        else:
            N, K = _log(rng, 512, 8192), _log(rng, 512, 8192)
            M = min(_log(rng, 1, 4096), 4096 * 8192 * 7168 // (N * K))
        if rng.random() < 0.5:  # half of them whole blocks wide, as most models' are
            N, K = N // 128 * 128, K // 128 * 128
        return _product(kind, M, N, K, E, spare, wide=kind == "dw" and rng.random() < 0.5)
    kind = rng.choice(["fwd", "bwd", "bwd8"])
    H = _log(rng, 256, 8192)
    if kind == "bwd8" or rng.random() < 0.5:
        H = H // 128 * 128
    if kind != "bwd8":
        E, spare = 0, 0.0
    return _glu(kind, min(_log(rng, 1, 32768), (1 << 25) // H), H, rng.choice(list(ACTS)), E, spare)


# ---- inputs ----------------------------------------------------------------

def _padded(rows, cols, dtype, pad):
    """An empty matrix whose rows start on 16 bytes, as the package's are."""
    return torch.empty(rows, -(-cols // pad) * pad, dtype=dtype, device=DEVICE)[:, :cols]


def _values(g, rows, cols, scale=1.0):
    """Activations: N(0, 1) in rows of different sizes, one value in a thousand large."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    x = x * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEVICE)) * scale
    x = torch.where(torch.rand(rows, cols, generator=g, device=DEVICE) < 1e-3, x * 20.0, x)
    return _padded(rows, cols, BF, 8).copy_(x)


def _weights(g, E, N, K):
    shape = (E, N, K) if E else (N, K)
    w = torch.randn(shape, generator=g, device=DEVICE) / math.sqrt(K)
    buf = torch.empty(*shape[:-1], -(-K // 8) * 8, dtype=BF, device=DEVICE)[..., :K]
    return buf.copy_(w)


def _counts(g, M, E, spare):
    """Rows of each expert, uneven as a router's are, one of them without any; `spare` of the rows belong to none."""
    if not E:
        return None
    used = M - int(M * spare)
    p = torch.rand(E, generator=g, device=DEVICE, dtype=F64).cpu() + 0.25
    p[E // 3] = 0.0
    ends = (torch.cumsum(p, 0) / p.sum() * used).round().to(torch.int64)
    ends[-1] = used
    return [0] + ends.tolist()


def _codes(g, rows, cols):
    """E4M3 codes of a quantised matrix."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE) * 120.0
    return _padded(rows, cols, F8, 16).copy_(x.clamp_(-TOP, TOP).to(F8))


def _scales(g, *shape):
    return torch.exp(0.5 * torch.randn(*shape, generator=g, device=DEVICE)) / 120.0


def _blocks(n):
    return -(-n // BLOCK)


def _column_blocks(M, ends):
    """(block, first row, last row) of the column form, and its number of blocks."""
    if ends is None:
        return [(b, b * BLOCK, min(M, (b + 1) * BLOCK)) for b in range(_blocks(M))], _blocks(M)
    out = []
    for e in range(len(ends) - 1):
        for i, r in enumerate(range(ends[e], ends[e + 1], BLOCK)):
            out.append((ends[e] // BLOCK + e + i, r, min(ends[e + 1], r + BLOCK)))
    return out, M // BLOCK + len(ends) - 1


def _row_index(M, ends):
    """The row at each place of the column form, M where it is zeros."""
    blocks, count = _column_blocks(M, ends)
    at = torch.full((count * BLOCK,), M, dtype=torch.int64)
    for b, r0, r1 in blocks:
        at[b * BLOCK:b * BLOCK + r1 - r0] = torch.arange(r0, r1)
    return at.to(DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    st = dict(case=dict(case), ends=_counts(g, case["M"], case["E"], case["spare"]) if case.get("mode") != "weights" else None)
    M, E, ends = case["M"], case["E"], st["ends"]
    st["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEVICE) if ends else None
    st["at"] = None
    if case["op"] == "quant":
        if case["mode"] == "weights":
            st["x"] = _weights(g, E, M, case["K"])
        elif case["mode"] == "again":
            st["x"] = dict(q=_codes(g, M, case["K"]), s=_scales(g, _blocks(case["K"]), M))
        else:
            st["x"] = _values(g, M, case["K"])
        if case["mode"] in ("both", "again"):
            st["at"] = _row_index(M, ends)
    elif case["op"] == "product":
        N, K = case["N"], case["K"]
        if case["kind"] == "dw":
            count = _column_blocks(M, ends)[1]
            at = _row_index(M, ends)
            for name, n in (("dy", N), ("x", K)):
                q = _codes(g, count * BLOCK, n)
                q.view(torch.uint8).masked_fill_((at == M)[:, None], 0)
                st[name] = dict(qc=q, sc=_scales(g, count, n) * 1e-2)
        else:
            depth = K if case["kind"] == "fwd" else N
            st["x"] = dict(q=_codes(g, M, depth), s=_scales(g, _blocks(depth), M))
            q = _codes(g, max(E, 1) * N, K)
            st["w"] = dict(q=q.view(E, N, K) if E else q, s=_scales(g, *((E,) if E else ()), _blocks(N), _blocks(K)) / math.sqrt(depth))
    else:
        H = case["H"]
        if case["kind"] == "fwd":
            both = _padded(M, 2 * H, BF, 8) if H % 8 == 0 else None
            st["gate"], st["up"] = _values(g, M, H), _values(g, M, H)
            if both is not None:  # the two halves of a projection's result
                both[:, :H], both[:, H:] = st["gate"], st["up"]
                st["gate"], st["up"] = both[:, :H], both[:, H:]
        else:
            st["gate"] = dict(q=_codes(g, M, H), s=_scales(g, _blocks(H), M))
            st["up"] = dict(q=_codes(g, M, H), s=_scales(g, _blocks(H), M))
            st["dh"] = _values(g, M, H, 0.1)
            if case["kind"] == "bwd8":
                st["at"] = _row_index(M, ends)
    return st


# ---- plain forms -----------------------------------------------------------

def _fit(v, a):
    """Codes of values whose block maxima are `a`, and the scales."""
    a = a.clamp_min(LEAST)
    return (v * TOP / a).to(F8), a / TOP


def _spread(s, n):
    """Scales [blocks, rows] for the n columns of the rows, [rows, n]."""
    return s.t().repeat_interleave(BLOCK, 1)[:, :n]


def _plain_rows(x):
    M, K = x.shape
    v = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(M, -1, BLOCK)
    q, s = _fit(v, v.abs().amax(2, keepdim=True))
    return dict(q=q.view(M, -1)[:, :K], s=s[:, :, 0].t().contiguous())


def _plain_cols(x, at):
    v = torch.cat([x, x.new_zeros(1, x.shape[1])])[at].view(-1, BLOCK, x.shape[1])
    q, s = _fit(v, v.abs().amax(1, keepdim=True))
    return dict(qc=q.view(-1, x.shape[1]), sc=s[:, 0])


def _plain_weight(w):
    N, K = w.shape[-2:]
    v = torch.nn.functional.pad(w.float(), (0, -K % BLOCK, 0, -N % BLOCK))
    v = v.view(*w.shape[:-2], _blocks(N), BLOCK, _blocks(K), BLOCK)
    q, s = _fit(v, v.abs().amax((-3, -1), keepdim=True))
    return dict(q=q.view(*w.shape[:-2], _blocks(N) * BLOCK, -1)[..., :N, :K], s=s[..., 0, :, 0])


def _plain_kept(x):
    return x["q"].float() * _spread(x["s"], x["q"].shape[1])


def _plain_w(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _plain_product(st):
    case, x, w, ends = st["case"], _plain_kept(st["x"]), st["w"], st["ends"]
    forward = case["kind"] == "fwd"
    if ends is None:
        wf = _plain_w(w["q"], w["s"])
        return (x @ (wf.t() if forward else wf)).to(BF)
    y = torch.zeros(case["M"], case["N" if forward else "K"], dtype=BF, device=DEVICE)
    for e in range(case["E"]):
        if ends[e] < ends[e + 1]:
            wf = _plain_w(w["q"][e], w["s"][e])
            y[ends[e]:ends[e + 1]] = (x[ends[e]:ends[e + 1]] @ (wf.t() if forward else wf)).to(BF)
    return y


def _plain_dw(st):
    case, ends = st["case"], st["ends"]
    dy, x = (st[n]["qc"].float() * st[n]["sc"].repeat_interleave(BLOCK, 0) for n in ("dy", "x"))
    to = F32 if case["wide"] else BF
    if ends is None:
        return (dy.t() @ x).to(to)
    out = torch.zeros(case["E"], case["N"], case["K"], dtype=to, device=DEVICE)
    for e in range(case["E"]):
        b0 = ends[e] // BLOCK + e
        b1 = b0 + _blocks(ends[e + 1] - ends[e])
        if b0 < b1:
            out[e] = (dy[b0 * BLOCK:b1 * BLOCK].t() @ x[b0 * BLOCK:b1 * BLOCK]).to(to)
    return out


def _act(name, x):
    """act(x) and act'(x)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * c * (x + 0.044715 * x ** 3)))
        return x * s, s + x * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * x * x)
    if name == "relu":
        return x * (x > 0), (x > 0).to(x.dtype)
    if name == "identity":
        return x, torch.ones_like(x)
    cdf = 0.5 * torch.erfc(-x / math.sqrt(2))
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)


def _plain_glu(st):
    case = st["case"]
    if case["kind"] == "fwd":
        gate, up = st["gate"].float(), st["up"].float()
        return dict(h=_plain_rows(_act(case["act"], gate)[0] * up), gate=_plain_rows(gate), up=_plain_rows(up))
    gate, up, dh = _plain_kept(st["gate"]), _plain_kept(st["up"]), st["dh"].float()
    a, d = _act(case["act"], gate)
    out, h = torch.cat([dh * up * d, dh * a], 1), a * up
    if case["kind"] == "bwd":
        return dict(d=out.to(BF), h=h.to(BF))
    return dict(d={**_plain_rows(out), **_plain_cols(out, st["at"])}, h=_plain_cols(h, st["at"]))


def _plain(st):
    case = st["case"]
    if case["op"] == "product":
        return _plain_dw(st) if case["kind"] == "dw" else _plain_product(st)
    if case["op"] == "glu":
        return _plain_glu(st)
    if case["mode"] == "weights":
        return _plain_weight(st["x"])
    if case["mode"] == "again":
        return _plain_cols(_plain_kept(st["x"]), st["at"])
    x = st["x"].float()
    out = _plain_rows(x)
    if case["mode"] == "both":
        out.update(_plain_cols(x, st["at"]))
    return out


# ---- the package's calls ---------------------------------------------------

def _given(out):
    """What a call returned, without what it was not asked for."""
    if not isinstance(out, dict):
        return out
    return {k: _given(v) for k, v in out.items() if v is not None}


def _own(st):
    import fp4_quant_gb300 as G
    case, offsets = st["case"], st["offsets"]
    if case["op"] == "quant":
        if case["mode"] == "weights":
            return _given(G.quant8_weight(st["x"]))
        mode = case["mode"]
        return _given(G.quant8(st["x"], rows=mode != "again", cols=mode != "rows", offsets=offsets if mode != "rows" else None))
    if case["op"] == "product":
        if case["kind"] == "dw":
            return G.linear8_dw(st["dy"], st["x"], offsets=offsets, dtype=F32 if case["wide"] else BF)
        return (G.linear8 if case["kind"] == "fwd" else G.linear8_dx)(st["x"], st["w"], offsets=offsets)
    act = ACTS[case["act"]]
    if case["kind"] == "fwd":
        return _given(G.glu8(st["gate"], st["up"], act=act))
    return _given(G.glu8_bwd(st["gate"], st["up"], st["dh"], act=act, quant=case["kind"] == "bwd8", offsets=offsets))


def run(state):
    return _own(state) if own else _plain(state)


# ---- work ------------------------------------------------------------------

def work(case):
    M, E = case["M"], case["E"]
    if case["op"] == "quant":
        K, mode = case["K"], case["mode"]
        if mode == "weights":
            n = max(E, 1) * M * K
            return {"bytes": 3 * n + max(E, 1) * _blocks(M) * _blocks(K) * 4, "flops": 2 * n}
        rows, cols = M * K + 4 * M * _blocks(K), M * K + 4 * K * (_blocks(M) if not E else M // BLOCK + E)
        if mode == "again":
            return {"bytes": rows + cols, "flops": 3 * M * K}
        return {"bytes": 2 * M * K + rows + (cols if mode == "both" else 0), "flops": (4 if mode == "both" else 2) * M * K}
    if case["op"] == "product":
        N, K = case["N"], case["K"]
        used = min(max(E, 1), M) * N * K  # experts with rows
        if case["kind"] == "dw":
            blocks = _blocks(M) if not E else M // BLOCK + E
            return {"bytes": M * (N + K) + 4 * blocks * (N + K) + max(E, 1) * N * K * (4 if case["wide"] else 2), "flops": 2 * M * N * K}
        depth, width = (K, N) if case["kind"] == "fwd" else (N, K)
        return {"bytes": M * depth + 4 * M * _blocks(depth) + used + 4 * used // BLOCK ** 2 + 2 * M * width, "flops": 2 * M * N * K}
    H = case["H"]
    kept = 2 * M * H + 8 * M * _blocks(H)
    if case["kind"] == "fwd":
        return {"bytes": 4 * M * H + kept + M * H + 4 * M * _blocks(H), "flops": 12 * M * H}
    if case["kind"] == "bwd":
        return {"bytes": kept + 2 * M * H + 6 * M * H, "flops": 16 * M * H}
    blocks = _blocks(M) if not E else M // BLOCK + E
    return {"bytes": kept + 2 * M * H + kept + 3 * (M * H + 4 * blocks * H), "flops": 24 * M * H}


# ---- the definitions in 64 bits --------------------------------------------

def _e4m3(v):
    """The E4M3 value nearest to v, ties to even: four significant bits, 2^-9 the least step."""
    m, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _blocked(v, rows, cols):
    """Codes and scales of a fp64 matrix in blocks of rows x cols."""
    R, C = v.shape
    p = v.new_zeros(-(-R // rows) * rows, -(-C // cols) * cols)
    p[:R, :C] = v
    p = p.view(-1, rows, p.shape[1] // cols, cols)
    a = p.abs().amax((1, 3)).clamp_min(LEAST)
    q = _e4m3(p * TOP / a[:, None, :, None])  # the product is exact for bf16 values: a tie stays one
    return q.reshape(-1, p.shape[2] * cols)[:R, :C], a / TOP


def _kept64(x):
    q = x["q"].to(F64)
    return q * x["s"].to(F64).t()[:, torch.arange(q.shape[1], device=DEVICE) // BLOCK]


def _rows64(v):
    q, s = _blocked(v, 1, BLOCK)
    return dict(q=q, s=s.t().contiguous())


def _cols64(v, ends):
    blocks, count = _column_blocks(v.shape[0], ends)
    p = v.new_zeros(count * BLOCK, v.shape[1])
    for b, r0, r1 in blocks:
        p[b * BLOCK:b * BLOCK + r1 - r0] = v[r0:r1]
    q, s = _blocked(p, BLOCK, 1)
    return dict(qc=q, sc=s)


def _act64(name, x):
    if name == "silu":
        s, z = torch.sigmoid(x), torch.sigmoid(-x)
        return x * s, s + x * s * z
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = 2 * c * (x + 0.044715 * x * x * x)
        s, z = torch.sigmoid(t), torch.sigmoid(-t)
        return x * s, s + x * s * z * 2 * c * (1 + 0.134145 * x * x)
    if name == "relu":
        return x.clamp_min(0), (x > 0).to(F64)
    if name == "identity":
        return x, torch.ones_like(x)
    phi = torch.special.ndtr(x)
    return x * phi, phi + x * torch.exp(-x * x / 2) * math.sqrt(0.5 / math.pi)


def exact(case, seed):
    st = prepare(case, seed)
    M, E, ends = case["M"], case["E"], st["ends"]
    if case["op"] == "quant":
        if case["mode"] == "weights":
            out = [_blocked(w.to(F64), BLOCK, BLOCK) for w in (st["x"] if E else st["x"][None])]
            q, s = (torch.stack(t) if E else t[0] for t in zip(*out))
            return dict(q=q, s=s)
        if case["mode"] == "again":
            return _cols64(_kept64(st["x"]), ends)
        v = st["x"].to(F64)
        return {**_rows64(v), **(_cols64(v, ends) if case["mode"] == "both" else {})}
    if case["op"] == "product":
        N, K = case["N"], case["K"]
        spans = [(e, ends[e], ends[e + 1]) for e in range(E)] if E else [(0, 0, M)]
        if case["kind"] == "dw":
            dy, x = (st[n]["qc"].to(F64).view(-1, BLOCK, w) * st[n]["sc"].to(F64)[:, None] for n, w in (("dy", N), ("x", K)))
            out = torch.zeros(max(E, 1), N, K, dtype=F64, device=DEVICE)
            for e, r0, r1 in spans:
                b = r0 // BLOCK + e
                n = _blocks(r1 - r0)
                out[e] = dy[b:b + n].reshape(-1, N).t() @ x[b:b + n].reshape(-1, K)
            return out if E else out[0]
        x = _kept64(st["x"])
        out = torch.zeros(M, N if case["kind"] == "fwd" else K, dtype=F64, device=DEVICE)
        row, col = torch.arange(N, device=DEVICE) // BLOCK, torch.arange(K, device=DEVICE) // BLOCK
        for e, r0, r1 in spans:
            q, s = (st["w"]["q"][e], st["w"]["s"][e]) if E else (st["w"]["q"], st["w"]["s"])
            w = q.to(F64) * s.to(F64)[row][:, col]
            out[r0:r1] = x[r0:r1] @ (w.t() if case["kind"] == "fwd" else w)
        return out
    if case["kind"] == "fwd":
        gate, up = st["gate"].to(F64), st["up"].to(F64)
        return dict(h=_rows64(_act64(case["act"], gate)[0] * up), gate=_rows64(gate), up=_rows64(up))
    gate, up, dh = _kept64(st["gate"]), _kept64(st["up"]), st["dh"].to(F64)
    a, d = _act64(case["act"], gate)
    out, h = torch.cat([dh * up * d, dh * a], 1), a * up
    if case["kind"] == "bwd":
        return dict(d=out, h=h)
    return dict(d={**_rows64(out), **_cols64(out, ends)}, h=_cols64(h, ends))
