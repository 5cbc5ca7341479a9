"""The experts of a transformer block in 8 bits, forward and backward: sorted rows
through the gated feed-forward layer of their expert, with every product's operands
in E4M3 with a scale per block of 128, and the backward from what the forward kept
in 8 bits (its input, gate and up: 1 byte per value, no bf16 activation).

    python examples/expert_ffn8.py            # needs a GB300 and the built library

``forward`` and ``backward`` launch on the current stream and wait for nothing.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp4_quant_gb300 as G  # noqa: E402


def make_weights(D, H, E, *, seed=0, device="cuda"):
    """bf16 weights of E experts: up [E, 2 H, D] (gates, then ups) and down [E, D, H]."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rnd(*shape, scale):
        return (scale * torch.randn(*shape, generator=g, device=device)).to(torch.bfloat16)

    return {"up": rnd(E, 2 * H, D, scale=D ** -0.5), "down": rnd(E, D, H, scale=H ** -0.5)}


def quantise(w):
    """The weights' 8-bit forms, made once per optimiser step."""
    return {k: G.quant8_weight(v) for k, v in w.items()}


def forward(xs, w8, offsets, *, act=G.ACT_SILU):
    """(y, saved): ``xs`` [R, D] bf16 sorted by expert (``G.dispatch``'s rows)."""
    H = w8["down"]["q"].shape[2]
    x8 = G.quant8(xs)
    u = G.linear8(x8, w8["up"], offsets=offsets)
    a = G.glu8(u[:, :H], u[:, H:], act=act)
    return G.linear8(a["h"], w8["down"], offsets=offsets), dict(x8={"q": x8["q"], "s": x8["s"]}, gate=a["gate"], up=a["up"], act=act)


def backward(dy, w8, s, offsets):
    """Gradients of xs and of the weights (fp32) from that of y."""
    dy8 = G.quant8(dy, cols=True, offsets=offsets)
    dh = G.linear8_dx(dy8, w8["down"], offsets=offsets)
    b = G.glu8_bwd(s["gate"], s["up"], dh, act=s["act"], quant=True, offsets=offsets)
    x8 = G.quant8(s["x8"], rows=False, cols=True, offsets=offsets)
    return {"xs": G.linear8_dx(b["d"], w8["up"], offsets=offsets),
            "up": G.linear8_dw(b["d"], x8, offsets=offsets, dtype=torch.float32),
            "down": G.linear8_dw(dy8, b["h"], offsets=offsets, dtype=torch.float32)}


def main():
    R, D, H, E = 32768, 2048, 1024, 64
    w8 = quantise(make_weights(D, H, E))
    xs, dy = (torch.randn(R, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    route = G.route(torch.randint(0, E, (R, 1), device="cuda"), E)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for _ in range(3):
        t[0].record()
        y, s = forward(xs, w8, route["offsets"])
        t[1].record()
        g = backward(dy, w8, s, route["offsets"])
        t[2].record()
    torch.cuda.synchronize()
    print(f"{R} rows, {E} experts: forward {t[0].elapsed_time(t[1]):.2f} ms, backward {t[1].elapsed_time(t[2]):.2f} ms, "
          f"|y| {float(y.float().norm()):.1f}, |dx| {float(g['xs'].float().norm()):.1f}")


if __name__ == "__main__":
    main()
