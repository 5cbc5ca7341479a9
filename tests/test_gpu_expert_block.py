"""The example's block, all the operators together, against autograd in 64 bits
on the same routing."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import expert_block as X  # noqa: E402


def _reference(x, w, ids, alpha, dy, dr):
    t = {k: v.double().requires_grad_(True) for k, v in {**w, "x": x}.items()}

    def rms(v, weight):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * weight

    n = rms(t["x"], t["norm_in"])
    p = torch.softmax(torch.gather(n @ t["router"].t(), 1, ids), 1)
    H = w["down"].shape[2]
    m = torch.zeros_like(t["x"])
    for e in range(w["router"].shape[0]):
        rows, k = (ids == e).nonzero(as_tuple=True)
        u = n[rows] @ t["up"][e].t() + t["up_bias"][e]
        f = (torch.nn.functional.silu(u[:, :H]) * u[:, H:]) @ t["down"][e].t()
        m = m.index_add(0, rows, f * p[rows, k][:, None])
    r = t["x"] + alpha * t["gate"] * rms(m, t["norm_out"])
    y = rms(r, t["norm_next"])
    ((y * dy.double()).sum() + (r * dr.double()).sum()).backward()
    return r.detach(), y.detach(), {k: v.grad for k, v in t.items()}


@pytest.mark.parametrize("T,D,H,E,k,alpha", [(1, 64, 32, 4, 2, 1.0), (77, 264, 136, 6, 2, 0.5), (500, 512, 256, 16, 4, 1.0)])
def test_block_forward_and_backward(T, D, H, E, k, alpha):
    w = X.make_weights(D, H, E, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x, dy, dr = (torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    r, y, s = X.forward(x, w, k, alpha=alpha)
    got = X.backward(dy, dr, w, s)
    want_r, want_y, want = _reference(x, w, s["ids"], alpha, dy, dr)
    # at most twelve roundings to bf16 one behind the other, 2^-9 each at worst
    # relative to the norm of what they round, and as much again through the
    # products of two rounded factors: 24 * 2^-9 = 0.047
    for name, a, b in [("r", r, want_r), ("y", y, want_y)] + [(n, got[n], want[n]) for n in got]:
        err = float((a.double() - b).norm() / b.norm())
        assert err < 0.047, (name, err)


def test_one_expert_for_all_and_experts_without_tokens():
    w = X.make_weights(128, 64, 8, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy, dr = (torch.randn(40, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    ids = torch.zeros(40, 2, dtype=torch.int64, device="cuda")
    ids[:, 1] = 5
    r, y, s = X.forward(x, w, 2, ids=ids)
    got = X.backward(dy, dr, w, s)
    want_r, want_y, want = _reference(x, w, ids, 1.0, dy, dr)
    for name, a, b in [("r", r, want_r), ("y", y, want_y)] + [(n, got[n], want[n]) for n in got]:
        assert float((a.double() - b).norm() / b.norm()) < 0.047, name
    idle = [e for e in range(8) if e not in (0, 5)]
    assert bool((got["up"][idle] == 0).all()) and bool((got["down"][idle] == 0).all()) and bool((got["up_bias"][idle] == 0).all())
