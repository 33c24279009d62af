"""README's training block, run as it is printed there, against float64 autograd of the
whole block: norm, router, experts, weighted sum, and the residual stream."""

import os
import re

import pytest
import torch

from moe_testlib import log
from ops_testlib import gen, half, randn

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
STEP = half(torch.bfloat16)


def block():
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), flags=re.S) if "moe_unpermute_backward" in b]
    assert len(blocks) == 1
    return blocks[0]


def close(got, ref, handoffs, what):
    """2-norm distance: each of `handoffs` roundings to bf16 on the way moves every value
    by at most half a step, 2^-8 of it; a factor 2 covers the sums that cancel."""
    got, ref = got.double(), ref.double()
    off = float((got - ref).norm() / ref.norm())
    assert off <= 2 * handoffs * STEP, (what, off, 2 * handoffs * STEP)


@pytest.mark.parametrize("M,H,I,E,k", [(200, 256, 128, 8, 2), (700, 520, 264, 16, 4)])
def test_training_block(M, H, I, E, k):
    import mixture_experts_routing_align_amd as moe

    log(f"README block M={M} H={H} I={I} E={E} top_k={k}")
    g = gen(M + H)
    v = dict(x=randn(g, M, H), res=randn(g, M, H), norm_w=randn(g, H, scale=0.1) + 1.0, router_w=randn(g, E, H, scale=H ** -0.5),
             gate=randn(g, E, I, H, scale=H ** -0.5), up=randn(g, E, I, H, scale=H ** -0.5), down=randn(g, E, H, I, scale=I ** -0.5),
             dout=randn(g, M, H), dz_stream=randn(g, M, H, scale=0.1))
    got = dict(v, torch=torch, moe=moe, E=E, k=k)
    exec(block(), got)
    torch.cuda.synchronize()

    names = ["res", "norm_w", "router_w", "gate", "up", "down"]
    leaf = {n: v[n].double().requires_grad_() for n in names}
    z = v["x"].double() + leaf["res"]
    n = z * (z.square().mean(1, keepdim=True) + 1e-6).pow(-0.5) * leaf["norm_w"]
    ids = got["ids"]
    wts = torch.softmax((n @ leaf["router_w"].T).gather(1, ids), 1)
    out = torch.zeros_like(z)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a = n[t]
        h = torch.nn.functional.silu(a @ leaf["gate"][e].T) * (a @ leaf["up"][e].T)
        out = out.index_add(0, t, wts[t, j, None] * (h @ leaf["down"][e].T))
    total = (out * v["dout"].double()).sum() + (z * v["dz_stream"].double()).sum()
    ref = dict(zip(names, torch.autograd.grad(total, [leaf[n] for n in names])))
    # z, n, h, y, out, and the weights from the rounded n
    close(got["out"], out.detach(), 6, "out")
    # those, and dy, dh, dz, dxs, the products' own roundings on the way back
    close(got["ddown"], ref["down"], 7, "down")
    close(got["dgate"], ref["gate"], 9, "gate")
    close(got["dup"], ref["up"], 9, "up")
    # z, n, h, y, the weights, dlogits, and the gradient itself, which reads n again
    close(got["drouter_w"], ref["router_w"], 8, "router")
    # both ways to n: ten roundings through the experts; the weights, dlogits, its product
    # and the sum of the two through the router, which reads y
    close(got["dx"], ref["res"], 15, "input")
    close(got["dnorm_w"], ref["norm_w"], 15, "norm weight")
