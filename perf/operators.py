"""Timed cases of the operators around the gated activation: block norms, expert routing, linear layers.

Each case is one call that a program makes: the forward or the backward of

* the block norms, ``r = x + alpha * gate * P(branch)`` and ``y = N(r)`` (``N``, ``P``: RMS norms with weights);
* the routing of tokens to experts: ``route`` + ``dispatch``, ``combine``, and its gradient;
* ``linear``, ``y = act(x W^T + b) + residual``, dense or with one weight matrix per expert.

``run`` computes it in elementary torch operations in fp32, rounded once at the end (``own`` false), or by the
package's calls (``own`` true).  ``exact`` restates the definitions in fp64.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
ACTS = {"none": 3, "silu": 0, "gelu_tanh": 1, "relu": 2, "gelu_erf": 4}  # the package's ACT_* values


# ---- cases ----------------------------------------------------------------

def _norm(op, M, D, **kw):
    c = dict(op=op, M=M, D=D, stream="bf16", branch=True, post=True, gates=1, alpha=1.0, w_offset=0.0, wtype="bf16")
    c.update(kw)
    return c


def _route(op, T, K, E, D, **kw):
    c = dict(op=op, T=T, K=K, E=E, D=D, drop=0.0, residual=False)
    c.update(kw)
    return c


def _linear(op, M, N, K, **kw):
    c = dict(op=op, M=M, N=N, K=K, E=0, spare=0.0, act="none", bias=False, residual=False, keep_z=False, wtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # one token of a decoding step: the branch is added to the stream and normed for the next block
        dict(_norm("norm_fwd", 1, 4096), name="norm_fwd_one_token"),
        # a training batch of 8 sequences with a gate row each (conditioned block), residual stream in fp32
        dict(_norm("norm_fwd", 16384, 7168, stream="fp32", gates=8, alpha=0.5, w_offset=1.0), name="norm_fwd_batch_fp32_stream"),
        # its training backward in bf16 with a channel gate, ragged token count
        dict(_norm("norm_bwd", 8191, 8192, gates=1, wtype="fp32"), name="norm_bwd_train"),
        # decoding step of 64 sequences, 8 of 128 experts each
        dict(_route("dispatch", 64, 8, 128, 2048), name="dispatch_decode"),
        # training batch, a few assignments dropped by a capacity limit
        dict(_route("dispatch", 16384, 8, 128, 2048, drop=0.02), name="dispatch_train"),
        # the way back, added to the residual stream; ragged token count
        dict(_route("combine", 16383, 8, 128, 2048, residual=True), name="combine_train"),
        # gradient of the way back: rows for the experts and the router's weight gradients
        dict(_route("combine_bwd", 16384, 8, 64, 2048, drop=0.02), name="combine_bwd_train"),
        # down projection of one token: reading the weights is all there is
        dict(_linear("linear_fwd", 1, 7168, 8192, residual=True), name="linear_fwd_one_token"),
        # up projection with bias and activation of a training batch, pre-activation kept for the backward
        dict(_linear("linear_fwd", 4096, 8192, 7168, act="gelu_tanh", bias=True, keep_z=True), name="linear_fwd_train"),
        # its backward: dx, dw, db through the activation; ragged token count
        dict(_linear("linear_bwd", 4095, 8192, 7168, act="gelu_tanh", bias=True), name="linear_bwd_train"),
        # the experts' gate/up projection for a prefill batch: 32768 routed rows over 64 experts
        dict(_linear("linear_fwd", 32768, 2048, 2048, E=64), name="experts_fwd_prefill"),
        # its training backward
        dict(_linear("linear_bwd", 32768, 2048, 2048, E=64), name="experts_bwd_train"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "dispatch", "combine", "combine_bwd", "linear_fwd", "linear_bwd"])
    wtype = rng.choice(["bf16", "fp32"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 256, 8192)
        D = D // 16 * 16 + 8 if rng.random() < 0.5 else D
        M = min(_log(rng, 1, 16384), (1 << 26) // D)
        stream = rng.choice(["bf16", "fp32"])
        branch = rng.random() < 0.8
        gates = rng.choice([0, 1, 1, 4, M]) if branch else 0
        if gates > 1:
            M = -(-M // gates) * gates
        post = branch and rng.random() < 0.6
        return _norm(op, M, D, stream=stream, branch=branch, post=post, gates=gates, alpha=rng.choice([1.0, 0.5]),
                     w_offset=rng.choice([0.0, 1.0]), wtype=wtype)
    if op in ("dispatch", "combine", "combine_bwd"):
        E = rng.choice([8, 16, 64, 128, 257])
        K = rng.choice([1, 2, 4, 6, 8])
        D = _log(rng, 256, 4096)
        D = D // 16 * 16 + 8 if rng.random() < 0.5 else D
        T = min(_log(rng, 1, 16384), max(1, (1 << 28) // (K * D)))
        return _route(op, T, K, E, D, drop=rng.choice([0.0, 0.02, 0.3]), residual=rng.random() < 0.5)
    if rng.random() < 0.5:
        E = rng.choice([4, 8, 32, 64])
        N, K = _log(rng, 256, 2048), _log(rng, 256, 2048)
        M = _log(rng, 8, 16384)
    else:
        E = 0
        N, K = _log(rng, 512, 8192), _log(rng, 512, 8192)
        M = min(_log(rng, 1, 4096), 4095 * 8192 * 7168 // (N * K))
    if rng.random() < 0.5:  # half of them whole tiles wide, as most models' are
        N, K = N // 128 * 128 + 64, K // 128 * 128 + 64
    act = rng.choice(list(ACTS))
    return _linear(op, M, N, K, E=E, spare=rng.choice([0.0, 0.05]) if E else 0.0, act=act, bias=rng.random() < 0.5, residual=op == "linear_fwd" and rng.random() < 0.5,
                   keep_z=op == "linear_fwd" and act != "none" and rng.random() < 0.5, wtype=wtype)


# ---- inputs ----------------------------------------------------------------

def _padded(values, dtype):
    """A 2-D (or 3-D) tensor of these values whose rows start on 16 bytes, as the package's operands do."""
    n = values.shape[-1]
    buf = torch.zeros(*values.shape[:-1], -(-n // 8) * 8, dtype=dtype, device=values.device)
    buf[..., :n] = values.to(dtype)
    return buf[..., :n]


def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _expert_ids(T, K, E, drop, g):
    """Top-K experts of random router logits with a popularity bias; a share `drop` of the entries is -1."""
    logits = torch.randn(T, E, generator=g, device=DEVICE) + 0.5 * torch.randn(E, generator=g, device=DEVICE)
    ids = torch.topk(logits, K, dim=1).indices
    if drop:
        ids = torch.where(torch.rand(ids.shape, generator=g, device=DEVICE) < drop, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(torch.gather(logits, 1, ids.clamp(min=0)), dim=1).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    s = {"case": c}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        M, D, st, wt = c["M"], c["D"], _dtype(c["stream"]), _dtype(c["wtype"])
        # a residual stream has a few channels far above the others
        big = 1.0 + 20.0 * (torch.rand(D, generator=g, device=DEVICE) < 0.005).float()
        x = _padded(rnd(M, D) * big, st)
        s["x"] = x
        s["branch"] = _padded(rnd(M, D), torch.bfloat16) if c["branch"] else None
        s["gate"] = _padded(0.5 + 0.5 * rnd(c["gates"], D), torch.bfloat16) if c["gates"] else None
        s["w_pre"] = (1.0 - c["w_offset"] + 0.1 * rnd(D)).to(wt)
        s["w_post"] = (1.0 - c["w_offset"] + 0.1 * rnd(D)).to(wt) if c["post"] else None
        if c["op"] == "norm_bwd":
            s["dy"] = _padded(rnd(M, D), torch.bfloat16)
            s["dr"] = _padded(rnd(M, D), st)
            # what the forward saved; x stands for the stream r it wrote
            s["rstd_pre"] = torch.rsqrt(x.float().square().mean(1) + EPS)
            s["rstd_post"] = torch.rsqrt(s["branch"].float().square().mean(1) + EPS) if c["post"] else None
    elif c["op"] in ("dispatch", "combine", "combine_bwd"):
        T, K, D, E = c["T"], c["K"], c["D"], c["E"]
        s["ids"], s["weights"] = _expert_ids(T, K, E, c["drop"], g)
        R = T * K
        if c["op"] == "dispatch":
            s["x"] = _padded(rnd(T, D), torch.bfloat16)
        else:
            s["ys"] = _padded(rnd(R, D), torch.bfloat16)
            slot, src, offsets = _route_plain(s["ids"], E)
            s["route"] = {"slot": slot, "src": src, "offsets": offsets}
            s["residual"] = _padded(rnd(T, D), torch.bfloat16) if c["residual"] else None
            s["dout"] = _padded(rnd(T, D), torch.bfloat16) if c["op"] == "combine_bwd" else None
    else:
        M, N, K, E = c["M"], c["N"], c["K"], c["E"]
        s["x"] = _padded(rnd(M, K), torch.bfloat16)
        # expert by expert: the fp32 draw of a whole stack would be large
        if E:
            w = _padded(torch.empty(E, N, K, dtype=torch.bfloat16, device=DEVICE), torch.bfloat16)
            for e in range(E):
                w[e] = (rnd(N, K) * K ** -0.5).to(torch.bfloat16)
            share = torch.softmax(0.5 * rnd(E), 0).cpu().double()
            # rows of the tail that no expert has are those whose assignments were dropped
            cuts = [0] + [int(v) for v in (share.cumsum(0) * M * (1.0 - c["spare"])).round()]
            if not c["spare"]:
                cuts[-1] = M
            s["offsets"] = torch.tensor(cuts, dtype=torch.int32, device=DEVICE)
            s["most"] = max(b - a for a, b in zip(cuts, cuts[1:]))  # the longest expert's rows
        else:
            w = _padded(rnd(N, K) * K ** -0.5, torch.bfloat16)
            s["offsets"] = None
        s["w"] = w
        s["bias"] = (0.1 * (rnd(E, N) if E else rnd(N))).to(_dtype(c["wtype"])) if c["bias"] else None
        s["residual"] = _padded(rnd(M, N), torch.bfloat16) if c["residual"] else None
        if c["op"] == "linear_bwd":
            s["dy"] = _padded(rnd(M, N), torch.bfloat16)
            s["z"] = _padded(rnd(M, N), torch.bfloat16) if c["act"] != "none" else None
    return s


# ---- plain forms -------------------------------------------------------------

def _rms(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _gate_rows(gate, M):
    """The gate row of each of M rows (one, or none as 1)."""
    if gate is None:
        return 1.0
    g = gate.float()
    return g if g.shape[0] in (1, M) else g.repeat_interleave(M // g.shape[0], 0)


def _norm_fwd_plain(s):
    c = s["case"]
    r = s["x"].float()
    rstd_post = None
    if s["branch"] is not None:
        t = s["branch"].float()
        if s["w_post"] is not None:
            rp = _rms(t)
            t, rstd_post = t * rp * (s["w_post"].float() + c["w_offset"]), rp[:, 0]
        r = r + c["alpha"] * _gate_rows(s["gate"], c["M"]) * t
    rs = _rms(r)
    out = {"y": (r * rs * (s["w_pre"].float() + c["w_offset"])).to(torch.bfloat16), "rstd_pre": rs[:, 0], "rstd_post": rstd_post}
    if s["branch"] is not None:
        out["r"] = r.to(s["x"].dtype)
    return out


def _norm_bwd_plain(s):
    c, M = s["case"], s["case"]["M"]
    rs = s["rstd_pre"][:, None]
    rh = s["x"].float() * rs
    dy = s["dy"].float()
    g = dy * (s["w_pre"].float() + c["w_offset"])
    dR = s["dr"].float() + rs * (g - rh * (g * rh).mean(1, keepdim=True))
    out = {"dx": dR.to(s["x"].dtype), "dw_pre": (dy * rh).sum(0), "dbranch": None, "dw_post": None, "dgate": None}
    if s["branch"] is not None:
        t = s["branch"].float()
        dt = c["alpha"] * _gate_rows(s["gate"], M) * dR
        if s["w_post"] is not None:
            rp = s["rstd_post"][:, None]
            bh, w = t * rp, s["w_post"].float() + c["w_offset"]
            t, q = bh * w, dt * w
            out["dw_post"] = (dt * bh).sum(0)
            dbranch = rp * (q - bh * (q * bh).mean(1, keepdim=True))
        else:
            dbranch = dt
        out["dbranch"] = dbranch.to(torch.bfloat16)
        if s["gate"] is not None:
            n = s["gate"].shape[0]
            out["dgate"] = (c["alpha"] * t * dR).reshape(n, M // n, -1).sum(1)
    return out


def _route_plain(ids, E):
    T, K = ids.shape
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    slot = torch.where(key < E, place, torch.full_like(place, -1)).to(torch.int32).reshape(T, K)
    src = torch.where(torch.arange(order.numel(), device=ids.device) < offsets[E], order, torch.full_like(order, -1)).to(torch.int32)
    return slot, src, offsets


def _dispatch_plain(s):
    slot, src, offsets = _route_plain(s["ids"], s["case"]["E"])
    xs = s["x"].float()[src.clamp(min=0) // s["case"]["K"]] * (src >= 0)[:, None]
    return {"slot": slot, "src": src, "offsets": offsets, "xs": xs.to(torch.bfloat16)}


def _combine_plain(s):
    slot = s["route"]["slot"]
    rows = s["ys"].float()[slot.clamp(min=0)]
    w = torch.where(slot >= 0, s["weights"], torch.zeros_like(s["weights"]))
    out = (rows * w[:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _combine_bwd_plain(s):
    K, slot, src = s["case"]["K"], s["route"]["slot"], s["route"]["src"]
    at = src.clamp(min=0)
    d = s["dout"].float()
    w = torch.where(src >= 0, s["weights"].reshape(-1)[at], torch.zeros(1, device=at.device))
    dys = w[:, None] * d[at // K]
    dw = (s["ys"].float()[slot.clamp(min=0)] * d[:, None, :]).sum(2) * (slot >= 0)
    return {"dys": dys.to(torch.bfloat16), "dw": dw}


def _act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return torch.clamp(z, min=0.0) if name == "relu" else z


def _act_grad(name, z):
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        th = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * z * z)
    if name == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return (z > 0).to(z.dtype) if name == "relu" else torch.ones_like(z)


def _by_expert(s):
    """Rows as [E, most]: their places in the sorted order and whether there is one; each row's expert, place in it, and whether it has one."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)[None]
    there = at < off[1:, None]
    row = torch.arange(s["case"]["M"], device=off.device)
    has = row < off[-1]
    e = torch.searchsorted(off[1:].contiguous(), row, right=True).clamp(max=off.numel() - 2)
    return at.clamp(max=s["case"]["M"] - 1), there, e, torch.where(has, row - off[e], torch.zeros_like(row)), has[:, None]


def _linear_fwd_plain(s):
    x, w = s["x"].float(), s["w"].float()
    b = 0.0 if s["bias"] is None else s["bias"].float()
    if s["offsets"] is None:
        z = x @ w.t() + b
    else:
        at, there, e, i, has = _by_expert(s)
        z = torch.bmm(x[at] * there[:, :, None], w.transpose(1, 2))[e, i]
        if s["bias"] is not None:
            z = z + b[e]
        z = z * has
    y = _act(s["case"]["act"], z)
    if s["residual"] is not None:
        y = y + (s["residual"].float() if s["offsets"] is None else s["residual"].float() * has)
    return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if s["case"]["keep_z"] else None}


def _linear_bwd_plain(s):
    x, w, dz = s["x"].float(), s["w"].float(), s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["case"]["act"], s["z"].float())
    if s["offsets"] is None:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    else:
        at, there, e, i, has = _by_expert(s)
        dzp = dz[at] * there[:, :, None]
        dx = torch.bmm(dzp, w)[e, i] * has
        dw = torch.bmm(dzp.transpose(1, 2), x[at] * there[:, :, None])
        db = dzp.sum(1)
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16), "db": db if s["bias"] is not None else None}


_PLAIN = {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "dispatch": _dispatch_plain, "combine": _combine_plain,
          "combine_bwd": _combine_bwd_plain, "linear_fwd": _linear_fwd_plain, "linear_bwd": _linear_bwd_plain}


# ---- the package's calls ---------------------------------------------------------

def _run_own(s):
    import fp4_quant_gb300 as G
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        o = G.block_norm(s["x"], s["branch"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"], w_offset=c["w_offset"], eps=EPS)
        return {k: o[k] for k in ("y", "rstd_pre", "rstd_post", "r") if o[k] is not None}
    if op == "norm_bwd":
        return G.block_norm_bwd(s["x"], s["dy"], s["dr"], rstd_pre=s["rstd_pre"], w_pre=s["w_pre"], branch=s["branch"], rstd_post=s["rstd_post"],
                                w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"], w_offset=c["w_offset"])
    if op == "dispatch":
        route = G.route(s["ids"], c["E"])
        return {**route, "xs": G.dispatch(s["x"], route)}
    if op == "combine":
        return G.combine(s["ys"], s["route"], s["weights"], residual=s["residual"])
    if op == "combine_bwd":
        return G.combine_bwd(s["dout"], s["ys"], s["route"], s["weights"])
    act = ACTS[c["act"]]
    if op == "linear_fwd":
        return G.linear(s["x"], s["w"], bias=s["bias"], act=act, residual=s["residual"], offsets=s["offsets"], keep_z=c["keep_z"])
    return G.linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=act, offsets=s["offsets"], need_db=c["bias"])


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- work ----------------------------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, st = c["M"] * c["D"], 4 if c["stream"] == "fp32" else 2
        vec = c["D"] * ((4 if c["wtype"] == "fp32" else 2) * (2 if c["post"] else 1) + 2 * c["gates"])
        rstd = 4 * c["M"] * (2 if c["post"] else 1)
        if op == "norm_fwd":
            return {"bytes": n * (st + 2 + ((2 + st) if c["branch"] else 0)) + vec + rstd, "flops": n * (12 if c["branch"] else 5)}
        grads = 4 * c["D"] * (1 + (1 if c["post"] else 0) + c["gates"])
        return {"bytes": n * (3 * st + 2 + (4 if c["branch"] else 0)) + vec + rstd + grads, "flops": n * (30 if c["branch"] else 12)}
    if op in ("dispatch", "combine", "combine_bwd"):
        T, K, D = c["T"], c["K"], c["D"]
        R = T * K
        kept = R * (1.0 - c["drop"])
        if op == "dispatch":  # int64 ids in; slots, sources, offsets and every row of xs out
            return {"bytes": 2 * D * (T + R) + 16 * R + 4 * (c["E"] + 1), "flops": 0}
        if op == "combine":
            return {"bytes": int(2 * D * (kept + T * (2 if c["residual"] else 1))) + 8 * R, "flops": int(2 * kept * D)}
        return {"bytes": int(2 * D * (T + kept + R)) + 16 * R, "flops": int(3 * kept * D)}
    M, N, K, E = c["M"], c["N"], c["K"], max(1, c["E"])
    hit = min(E, M)  # experts that have rows
    vec = (4 if c["wtype"] == "fp32" else 2) * hit * N if c["bias"] else 0
    if op == "linear_fwd":
        out = 1 + (1 if c["residual"] else 0) + (1 if c["keep_z"] else 0)
        return {"bytes": 2 * (M * K + hit * N * K + out * M * N) + vec, "flops": 2 * M * N * K}
    return {"bytes": 2 * (2 * M * K + hit * N * K + E * N * K + M * N * (2 if c["act"] != "none" else 1)) + (4 * E * N if c["bias"] else 0),
            "flops": 4 * M * N * K}


# ---- the definitions in 64 bits ----------------------------------------------------

def _d(t):
    return None if t is None else t.double()


def _exact_act(name, z, grad):
    """act or act' by the logistic function and the normal distribution, in fp64."""
    if name in ("silu", "gelu_tanh"):
        k = 2.0 * math.sqrt(2.0 / math.pi)
        u, du = (z, torch.ones_like(z)) if name == "silu" else (k * (z + 0.044715 * z ** 3), k * (1.0 + 0.134145 * z ** 2))
        p, q = 1.0 / (1.0 + torch.exp(-u)), 1.0 / (1.0 + torch.exp(u))
        return p * (1.0 + z * q * du) if grad else z * p
    if name == "gelu_erf":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return cdf + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi) if grad else z * cdf
    if name == "relu":
        return torch.where(z > 0, torch.ones_like(z) if grad else z, torch.zeros_like(z))
    return torch.ones_like(z) if grad else z


def _exact_norm(s, out, a, b):
    """Rows a..b of the norms (they are independent; gradients of vectors are added up in `out`)."""
    c = s["case"]
    x, branch = _d(s["x"][a:b]), None if s["branch"] is None else _d(s["branch"][a:b])
    D = c["D"]
    wp = _d(s["w_pre"]) + c["w_offset"]
    wq = None if s["w_post"] is None else _d(s["w_post"]) + c["w_offset"]
    gate_row = None if s["gate"] is None else torch.arange(a, b, device=x.device) // (c["M"] // c["gates"])
    gate = 1.0 if gate_row is None else _d(s["gate"])[gate_row]
    if c["op"] == "norm_fwd":
        r = x
        if branch is not None:
            if wq is not None:
                sq = (branch.pow(2).sum(1) / D + EPS).sqrt()
                out["rstd_post"][a:b] = 1.0 / sq
                branch = branch / sq[:, None] * wq
            r = x + c["alpha"] * branch * gate
            out["r"][a:b] = r
        sq = (r.pow(2).sum(1) / D + EPS).sqrt()
        out["rstd_pre"][a:b] = 1.0 / sq
        out["y"][a:b] = r / sq[:, None] * wp
        return
    rs = _d(s["rstd_pre"][a:b])[:, None]
    dy = _d(s["dy"][a:b])
    n = x * rs
    up = dy * wp
    total = _d(s["dr"][a:b]) + up * rs - n * rs * ((up * n).sum(1, keepdim=True) / D)
    out["dx"][a:b] = total
    out["dw_pre"] += (dy * n).sum(0)
    if branch is None:
        return
    down = total * gate * c["alpha"]
    if wq is None:
        scaled = branch
        out["dbranch"][a:b] = down
    else:
        rp = _d(s["rstd_post"][a:b])[:, None]
        n = branch * rp
        scaled = n * wq
        out["dw_post"] += (down * n).sum(0)
        up = down * wq
        out["dbranch"][a:b] = up * rp - n * rp * ((up * n).sum(1, keepdim=True) / D)
    if gate_row is not None:
        out["dgate"].index_add_(0, gate_row, total * scaled * c["alpha"])


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    f64 = dict(dtype=torch.float64, device=DEVICE)
    if op in ("norm_fwd", "norm_bwd"):
        M, D = c["M"], c["D"]
        keys = {"y": (M, D), "rstd_pre": (M,)} if op == "norm_fwd" else {"dx": (M, D), "dw_pre": (D,)}
        if c["branch"]:
            keys |= {"r": (M, D)} if op == "norm_fwd" else {"dbranch": (M, D)}
        if c["post"]:
            keys |= {"rstd_post": (M,)} if op == "norm_fwd" else {"dw_post": (D,)}
        if c["gates"] and op == "norm_bwd":
            keys |= {"dgate": (c["gates"], D)}
        out = {k: torch.zeros(*v, **f64) for k, v in keys.items()}
        for a in range(0, M, 4096):
            _exact_norm(s, out, a, min(M, a + 4096))
        return out
    if op in ("dispatch", "combine", "combine_bwd"):
        T, K = s["ids"].shape
        if op == "dispatch":  # counted expert by expert on the host
            lists = [[] for _ in range(c["E"])]
            for j, e in enumerate(s["ids"].reshape(-1).tolist()):
                if 0 <= e < c["E"]:
                    lists[e].append(j)
            offsets, src = [0], []
            for one in lists:
                src += one
                offsets.append(len(src))
            slot = torch.full((T * K,), -1, dtype=torch.int32)
            slot[torch.tensor(src, dtype=torch.long)] = torch.arange(len(src), dtype=torch.int32)
            xs = torch.zeros(T * K, c["D"], **f64)
            xs[:len(src)] = _d(s["x"])[torch.tensor(src, dtype=torch.long, device=DEVICE) // K]
            src = torch.tensor(src + [-1] * (T * K - len(src)), dtype=torch.int32)
            return {"slot": slot.reshape(T, K).to(DEVICE), "src": src.to(DEVICE), "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEVICE), "xs": xs}
        slot = s["route"]["slot"].long()
        if op == "combine":
            out = torch.zeros(T, c["D"], **f64) if s["residual"] is None else _d(s["residual"]).clone()
            for k in range(K):
                t = (slot[:, k] >= 0).nonzero()[:, 0]
                out[t] += _d(s["ys"][slot[t, k]]) * _d(s["weights"][t, k])[:, None]
            return out
        dys, dw = torch.zeros(T * K, c["D"], **f64), torch.zeros(T, K, **f64)
        for k in range(K):
            t = (slot[:, k] >= 0).nonzero()[:, 0]
            d = _d(s["dout"][t])
            dys[slot[t, k]] = d * _d(s["weights"][t, k])[:, None]
            dw[t, k] = (d * _d(s["ys"][slot[t, k]])).sum(1)
        return {"dys": dys, "dw": dw}
    M, N, K, E = c["M"], c["N"], c["K"], c["E"]
    cuts = [0, M] if not E else s["offsets"].tolist()  # rows past the last expert's stay zero
    stack = (lambda t, e: t[e]) if E else (lambda t, e: t)
    if op == "linear_fwd":
        z = torch.zeros(M, N, **f64)
        for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
            z[a:b] = _d(s["x"][a:b]) @ _d(stack(s["w"], e)).t()
            if s["bias"] is not None:
                z[a:b] += _d(stack(s["bias"], e))
        y = _exact_act(c["act"], z, False)
        if s["residual"] is not None:
            y[:cuts[-1]] += _d(s["residual"][:cuts[-1]])
        return {"y": y, "z": z if c["keep_z"] else None}
    dz = _d(s["dy"])
    if s["z"] is not None:
        dz = dz * _exact_act(c["act"], _d(s["z"]), True)
    dx, dw, db = torch.zeros(M, K, **f64), torch.zeros(max(E, 1), N, K, **f64), torch.zeros(max(E, 1), N, **f64)
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        dx[a:b] = dz[a:b] @ _d(stack(s["w"], e))
        dw[e] = dz[a:b].t() @ _d(s["x"][a:b])
        db[e] = dz[a:b].sum(0)
    if not E:
        dw, db = dw[0], db[0]
    return {"dx": dx, "dw": dw, "db": db if c["bias"] else None}
