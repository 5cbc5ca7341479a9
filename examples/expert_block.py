"""A transformer block's mixture of experts, forward and backward, from the
package's calls: the norms around it, the router's sort, the experts' products,
the gated activation between them, and the way back to the residual stream.

    python examples/expert_block.py            # needs a GB300 and the built library

``forward`` keeps what ``backward`` needs; both launch on the current stream and
wait for nothing.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp4_quant_gb300 as G  # noqa: E402


def make_weights(D, H, E, *, seed=0, device="cuda"):
    """Random weights of a block of width D with E experts of hidden width H."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rnd(*shape, scale):
        return (scale * torch.randn(*shape, generator=g, device=device)).to(torch.bfloat16)

    return {"norm_in": 1 + rnd(D, scale=0.1), "norm_out": 1 + rnd(D, scale=0.1), "norm_next": 1 + rnd(D, scale=0.1),
            "gate": rnd(D, scale=0.5), "router": rnd(E, D, scale=D ** -0.5),
            "up": rnd(E, 2 * H, D, scale=D ** -0.5), "up_bias": rnd(E, 2 * H, scale=0.1), "down": rnd(E, D, H, scale=H ** -0.5)}


def forward(x, w, k, *, alpha=1.0, ids=None):
    """(r, y, saved): the residual stream behind the block, its norm for the
    next one, and what ``backward`` needs.  ``x`` [T, D] bf16; each token goes to
    the k experts with the largest logits (or to ``ids``)."""
    T, H = x.shape[0], w["down"].shape[2]
    E = w["router"].shape[0]
    n = G.block_norm(x, w_pre=w["norm_in"])
    logits = G.linear(n["y"], w["router"])["y"].float()
    if ids is None:
        ids = torch.topk(logits, k, dim=1).indices.contiguous()
    p = torch.softmax(torch.gather(logits, 1, ids), dim=1).contiguous()
    route = G.route(ids, E)
    xs = G.dispatch(n["y"], route)
    u = G.linear(xs, w["up"], bias=w["up_bias"], offsets=route["offsets"])["y"]  # [T k, 2 H]: gates, then ups
    h = G.fwd(u[:, :H], u[:, H:], act=G.ACT_SILU, fmt=G.FMT_BF16)["out"]
    ys = G.linear(h, w["down"], offsets=route["offsets"])["y"]
    m = G.combine(ys, route, p)
    o = G.block_norm(x, m, w_post=w["norm_out"], w_pre=w["norm_next"], gate=w["gate"], alpha=alpha)
    saved = dict(x=x, n=n, ids=ids, p=p, route=route, xs=xs, u=u, h=h, ys=ys, m=m, o=o, alpha=alpha, T=T)
    return o["r"], o["y"], saved


def backward(dy, dr, w, s):
    """Gradients of x and of every weight from those of y and r."""
    H, route = w["down"].shape[2], s["route"]
    b = G.block_norm_bwd(s["o"]["r"], dy, dr, rstd_pre=s["o"]["rstd_pre"], w_pre=w["norm_next"], branch=s["m"], rstd_post=s["o"]["rstd_post"],
                         w_post=w["norm_out"], gate=w["gate"], alpha=s["alpha"])
    c = G.combine_bwd(b["dbranch"], s["ys"], route, s["p"])
    down = G.linear_bwd(c["dys"], s["h"], w["down"], offsets=route["offsets"])
    du = G.bwd(s["u"][:, :H], s["u"][:, H:], down["dx"], act=G.ACT_SILU, fmt=G.FMT_BF16)["out"]
    up = G.linear_bwd(du, s["xs"], w["up"], offsets=route["offsets"], need_db=True)
    dn = G.dispatch_bwd(up["dx"], route)
    # the router: through the softmax over the chosen logits
    E = w["router"].shape[0]
    dlogits = torch.zeros(s["T"], -(-E // 8) * 8, device=dn.device)  # rows start on 16 bytes
    dlogits.scatter_add_(1, s["ids"], s["p"] * (c["dw"] - (s["p"] * c["dw"]).sum(1, keepdim=True)))
    r = G.linear_bwd(dlogits.to(torch.bfloat16)[:, :E], s["n"]["y"], w["router"])
    a = G.block_norm_bwd(s["x"], (dn.float() + r["dx"].float()).to(torch.bfloat16), b["dx"], rstd_pre=s["n"]["rstd_pre"], w_pre=w["norm_in"])
    return {"x": a["dx"], "norm_in": a["dw_pre"], "norm_next": b["dw_pre"], "norm_out": b["dw_post"], "gate": b["dgate"][0],
            "router": r["dw"], "up": up["dw"], "up_bias": up["db"], "down": down["dw"]}


def main():
    T, D, H, E, k = 4096, 2048, 1024, 64, 8
    w = make_weights(D, H, E)
    x, dy, dr = (torch.randn(T, D, device="cuda").to(torch.bfloat16) for _ in range(3))
    for _ in range(3):
        _, _, s = forward(x, w, k)
        backward(dy, dr, w, s)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    t[0].record()
    r, y, s = forward(x, w, k)
    t[1].record()
    g = backward(dy, dr, w, s)
    t[2].record()
    torch.cuda.synchronize()
    print(f"{T} tokens, {E} experts, {k} each: forward {t[0].elapsed_time(t[1]):.2f} ms, backward {t[1].elapsed_time(t[2]):.2f} ms, "
          f"|y| {float(y.float().norm()):.1f}, |dx| {float(g['x'].float().norm()):.1f}")


if __name__ == "__main__":
    main()
