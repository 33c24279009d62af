"""Matrices whose byte offsets pass 32 bits: the last rows get the results of the
same rows in small matrices, bit for bit."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import gen

pytestmark = pytest.mark.gpu

ROWS, C = 270_000, 8192  # 4.4 GB of bf16
TAIL = 300


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.fixture(scope="module")
def x():
    t = torch.empty(ROWS, C, dtype=torch.bfloat16, device="cuda")
    t.normal_(generator=gen(1))
    yield t
    del t
    torch.cuda.empty_cache()


def test_norm(moe, x):
    log("norm of 270000 x 8192")
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    y, _, z, rstd = moe.moe_add_rms_norm(x, w, 1e-6, residual=x, save_rstd=True)
    dx, _ = moe.moe_add_rms_norm_backward(y, z, w, rstd, dz=x)
    s = x[-TAIL:].contiguous()
    y2, _, z2, rstd2 = moe.moe_add_rms_norm(s, w, 1e-6, residual=s, save_rstd=True)
    dx2, _ = moe.moe_add_rms_norm_backward(y2, z2, w, rstd2, dz=s)
    for a, b in ((y, y2), (z, z2), (rstd, rstd2), (dx, dx2)):
        assert torch.equal(a[-TAIL:], b)


def test_permute_and_back(moe, x):
    log("permute of 270000 rows")
    perm = torch.arange(ROWS - 1, -1, -1, dtype=torch.int32, device="cuda")  # one slot a token, reversed
    out, _ = moe.moe_permute(x, perm, 1, ROWS)
    assert torch.equal(out[-TAIL:], x[:TAIL].flip(0)) and torch.equal(out[:TAIL], x[-TAIL:].flip(0))
    back = moe.moe_unpermute(out, perm, 1)
    assert torch.equal(back[-TAIL:], x[-TAIL:]) and torch.equal(back[:TAIL], x[:TAIL])
    w = torch.ones(ROWS, 1, device="cuda")
    dy, _ = moe.moe_unpermute_backward(back, out, perm, w, dy=out)
    assert torch.equal(dy[-TAIL:], x[:TAIL].flip(0))


def test_products(moe, x):
    log("products of 270000 rows")
    N = 16
    w = (torch.randn(2, N, C, generator=gen(2), device="cuda") * C ** -0.5).to(torch.bfloat16)
    # two experts; the second one's run begins past 2^32 bytes
    split = ROWS - TAIL
    offsets = torch.tensor([0, split, ROWS], dtype=torch.int32, device="cuda")
    counts = torch.tensor([split, TAIL], dtype=torch.int32, device="cuda")
    s = x[split:].contiguous()
    one = (torch.tensor([0, TAIL], dtype=torch.int32, device="cuda"), torch.tensor([TAIL], dtype=torch.int32, device="cuda"))
    y, _, _ = moe.moe_grouped_linear(x, w, offsets, counts)
    # summed in whole chunks of 128 columns by either tile, so only the order may differ
    ref = s.double() @ w[1].double().T
    mag = s.double().abs() @ w[1].double().abs().T
    assert bool(((y[split:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (C + 8) * 2.0 ** -23 * mag).all())
    dw, _, _, _ = moe.moe_grouped_linear_backward_w(y, x, offsets, counts, dtype=torch.float32)
    dw2, _, _, _ = moe.moe_grouped_linear_backward_w(y[split:].contiguous(), s, *one, dtype=torch.float32)
    err = (dw[1].double() - dw2[0].double()).abs()
    bound = 2 * (TAIL + 8) * 2.0 ** -23 * (y[split:].double().abs().T @ s.double().abs())
    assert bool((err <= bound).all())
    dx = moe.moe_grouped_linear_backward_x(y, w, offsets, counts)
    ref = y[split:].double() @ w[1].double()
    mag = y[split:].double().abs() @ w[1].double().abs()
    assert bool(((dx[split:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (N + 8) * 2.0 ** -23 * mag + 1e-37).all())
