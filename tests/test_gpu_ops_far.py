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


# More workgroups than one grid dimension holds (2^21): the last rows again.

MANY = 2 ** 21


def test_many_rows_norm(moe):
    M, H = 4 * MANY + 37, 8  # four rows a workgroup
    log(f"norm of {M} x {H}")
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(3))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, _, _, rstd = moe.moe_add_rms_norm(x, w, 1e-6, save_rstd=True)
    for part in (slice(0, TAIL), slice(4 * MANY - TAIL, 4 * MANY + 37)):
        y2, _, _, rstd2 = moe.moe_add_rms_norm(x[part].contiguous(), w, 1e-6, save_rstd=True)
        assert torch.equal(y[part], y2) and torch.equal(rstd[part], rstd2)


@pytest.mark.parametrize("M,H", [(4 * MANY + 37, 8), (MANY + 37, 1032)])  # a wave, a workgroup per token
def test_many_rows_permute(moe, M, H):
    log(f"permute of {M} x {H}")
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(4))
    perm = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    out, _ = moe.moe_permute(x, perm, 1, M)
    assert torch.equal(out, x.flip(0))
    w = torch.full((M, 1), 0.5, device="cuda")
    assert torch.equal(moe.moe_unpermute(out, perm, 1, topk_weights=w), x * 0.5)  # halving rounds nothing here
    dy, dw = moe.moe_unpermute_backward(x, out, perm, w)
    assert torch.equal(dy, out * 0.5)
    for part in (slice(0, TAIL), slice(M - TAIL, M)):
        ref = x[part].double().square().sum(1)
        assert bool(((dw[part, 0].double() - ref).abs() <= (H + 8) * 2.0 ** -23 * ref).all())


def test_many_tiles(moe):
    # a workgroup per 16 rows in the activation's gradient
    rows, N = 16 * MANY + 333, 8
    log(f"activation gradient of {rows} x {N}")
    pre = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(5))
    dy = torch.empty_like(pre).normal_(generator=gen(6))
    dz = moe.moe_grouped_act_backward(dy, pre, "gelu")
    for part in (slice(0, TAIL), slice(rows - 2 * TAIL, rows)):
        assert torch.equal(dz[part], moe.moe_grouped_act_backward(dy[part].contiguous(), pre[part].contiguous(), "gelu"))
    del pre, dy, dz
    # a workgroup per 16 rows by 16 columns of each expert: 1024 experts of 32 rows
    E, N, K = 1024, 16400, 8
    log(f"few rows of {E} experts, {N} x {K}")
    rows = 32 * E
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(7))
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(8))
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 32
    counts = torch.full((E,), 32, dtype=torch.int32, device="cuda")
    y, _, _ = moe.moe_grouped_linear(x, w, offsets, counts)
    for e in (0, 511, 1022, 1023):
        one, _, _ = moe.moe_grouped_linear(x[32 * e:32 * e + 32].contiguous(), w[e:e + 1].contiguous(), offsets[:2], counts[:1])
        assert torch.equal(y[32 * e:32 * e + 32], one)
    xs = x.view(E, 32, K).float()
    for e0 in range(0, E, 64):  # every tile was taken
        ref = torch.stack([xs[e] @ w[e].float().T for e in range(e0, e0 + 64)])
        mag = torch.stack([xs[e].abs() @ w[e].float().abs().T for e in range(e0, e0 + 64)])
        got = y[32 * e0:32 * (e0 + 64)].view(64, 32, N).float()
        # half a bf16 step, and K + 8 float32 roundings on either side
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * (K + 8) * 2.0 ** -23 * mag).all())
