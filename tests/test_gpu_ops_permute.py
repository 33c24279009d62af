"""Rows laid out by expert and brought back, and the gradient, against indexing
in float64 (bounds: see ops_testlib)."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import (SUM, Routed, assert_untouched, assert_within, gen, half, poison, quantised, randn, untouched_buffer)

pytestmark = pytest.mark.gpu

CASES = [  # M, E, k, BS, H, mode, drop
    (1, 8, 2, 16, 2048, "random", 0.0),
    (1, 1, 1, 1, 8, "random", 0.0),
    (3, 5, 5, 4, 7, "random", 0.3),
    (8, 128, 8, 16, 2048, "random", 0.0),
    (33, 16, 3, 16, 1001, "skew", 0.2),
    (64, 300, 20, 1, 264, "random", 0.5),
    (129, 4, 2, 64, 4096, "one", 0.0),
    (2500, 32, 4, 16, 520, "skew", 0.1),
    (2300, 64, 9, 16, 2047, "random", 0.0),
    (2200, 16, 11, 16, 264, "random", 0.1),
    (40, 8, 2, 16, 256, "random", 1.0),  # every slot dropped
]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.mark.parametrize("M,E,k,BS,H,mode,drop", CASES)
def test_permute_and_back(moe, M, E, k, BS, H, mode, drop):
    log(f"permute M={M} E={E} k={k} BS={BS} H={H} {mode} drop={drop}")
    r = Routed(moe, M, E, k, BS, M + H, mode, drop)
    g = gen(M)
    x = randn(g, M, H)
    out = untouched_buffer(r.rows, H, dtype=torch.bfloat16)
    got, none = moe.moe_permute(x, r.perm, k, r.rows, out=out)
    torch.cuda.synchronize()
    assert none is None and got is out
    p = r.perm.long()
    slots = torch.nonzero(p >= 0)[:, 0]
    assert torch.equal(out[p[slots]], x[slots // k])
    assert_untouched(out, r.kept, "permute")

    y = poison(randn(g, r.rows, H), r.kept)
    rows = torch.zeros(M * k, H, dtype=torch.float64, device="cuda")
    rows[slots] = y[p[slots]].double()
    rows = rows.reshape(M, k, H)
    w = r.weights.double()[..., None]
    bf = half(torch.bfloat16)
    o = moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)
    ref = (rows * w).sum(1)
    assert_within(o, ref, bf * ref.abs() + (k + 1) * SUM * (rows * w).abs().sum(1) + 1e-37, "weighted")
    o = moe.moe_unpermute(y, r.perm, k)
    ref = rows.sum(1)
    assert_within(o, ref, bf * ref.abs() + (k + 1) * SUM * rows.abs().sum(1) + 1e-37, "plain")

    dout = randn(g, M, H)
    dy = untouched_buffer(r.rows, H, dtype=torch.bfloat16)
    _, dw = moe.moe_unpermute_backward(dout, y, r.perm, r.weights, dy=dy)
    torch.cuda.synchronize()
    prod = dout.double()[:, None] * rows
    assert_within(dw, prod.sum(2), (H / 64 + 16) * SUM * prod.abs().sum(2) + 1e-37, "dweights")
    ref = (w * dout.double()[:, None]).reshape(M * k, H)[slots]
    assert_within(dy[p[slots]], ref, (bf + 2 * SUM) * ref.abs() + 1e-37, "dy")
    assert_untouched(dy, r.kept, "unpermute backward")
    # over y's own buffer
    _, dw2 = moe.moe_unpermute_backward(dout, y, r.perm, r.weights, dy=y)
    assert torch.equal(dw2, dw) and torch.equal(y[r.kept], dy[r.kept])


@pytest.mark.parametrize("M,E,k,BS,H", [(1, 8, 2, 16, 128), (17, 16, 4, 16, 2048), (2100, 24, 3, 1, 384)])
def test_permute_8bit(moe, M, E, k, BS, H):
    r = Routed(moe, M, E, k, BS, M, "random", 0.1)
    codes, scale = quantised(randn(gen(M), M, H))
    out = untouched_buffer(r.rows, H, dtype=torch.float8_e4m3fn)
    out_scale = untouched_buffer(r.rows, H // 128, dtype=torch.float32)
    moe.moe_permute(codes, r.perm, k, r.rows, scale=scale, out=out, out_scale=out_scale)
    torch.cuda.synchronize()
    p = r.perm.long()
    slots = torch.nonzero(p >= 0)[:, 0]
    assert torch.equal(out.view(torch.uint8)[p[slots]], codes.view(torch.uint8)[slots // k])
    assert torch.equal(out_scale[p[slots]], scale[slots // k])
    assert_untouched(out, r.kept)
    assert_untouched(out_scale, r.kept)


def test_permute_past_the_caches(moe):
    """Sorted rows too large for the caches take stores of their own."""
    M, E, k, H = 2100, 16, 8, 6200
    r = Routed(moe, M, E, k, 1, 2)
    assert r.rows * H * 2 > 192 << 20
    x = randn(gen(1), M, H)
    out, _ = moe.moe_permute(x, r.perm, k, r.rows)
    torch.cuda.synchronize()
    p = r.perm.long()
    for lo in range(0, M * k, 4000):
        assert torch.equal(out[p[lo:lo + 4000]], x[torch.arange(lo, min(lo + 4000, M * k), device="cuda") // k])


def test_positions_out_of_range_are_skipped(moe):
    """Positions at or past the sorted matrix's height, or negative, name no row."""
    M, k, H, rows = 4, 2, 64, 6
    perm = torch.tensor([0, 5, 6, -1, 1, 2 ** 31 - 1, -2 ** 31, 3], dtype=torch.int32, device="cuda")
    x = randn(gen(0), M, H)
    out = untouched_buffer(rows, H, dtype=torch.bfloat16)
    moe.moe_permute(x, perm, k, rows, out=out)
    torch.cuda.synchronize()
    kept = torch.zeros(rows, dtype=torch.bool, device="cuda")
    kept[[0, 5, 1, 3]] = True
    assert torch.equal(out[[0, 5, 1, 3]], x[[0, 0, 2, 3]])
    assert_untouched(out, kept)
    o = moe.moe_unpermute(out, perm, k)
    w = torch.ones(M, k, device="cuda")
    _, dw = moe.moe_unpermute_backward(x, out, perm, w, dy=torch.zeros_like(out))
    torch.cuda.synchronize()
    assert torch.equal(o[2], x[2]) and torch.equal(o[3], x[3]) and not bool(o[1].any())
    assert not bool(dw[1].any()) and float(dw[2, 1]) == 0 and float(dw[3, 0]) == 0


def test_unpermute_is_the_gradient_of_permute(moe):
    """<permute(x), s> = <x, unpermute(s)> for rows of integers, exactly."""
    r = Routed(moe, 50, 8, 3, 16, 5, "random", 0.1)
    g = gen(2)
    x = torch.randint(-4, 5, (50, 96), generator=g, device="cuda").to(torch.bfloat16)
    s = torch.randint(-4, 5, (r.rows, 96), generator=g, device="cuda").to(torch.bfloat16)
    xs, _ = moe.moe_permute(x, r.perm, 3, r.rows, out=torch.zeros(r.rows, 96, dtype=torch.bfloat16, device="cuda"))
    back = moe.moe_unpermute(s, r.perm, 3)
    assert float((xs.double() * s.double()).sum()) == float((x.double() * back.double()).sum())


def test_graph_replay(moe):
    M, E, k, H = 300, 16, 4, 520
    r = Routed(moe, M, E, k, 16, 3)
    x, y, dout = randn(gen(1), M, H), randn(gen(2), r.rows, H), randn(gen(3), M, H)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    bufs = [torch.zeros(r.rows, H, dtype=torch.bfloat16, device="cuda") for _ in range(4)]

    def step(a, b):
        xs, _ = moe.moe_permute(x, r.perm, k, r.rows, out=a)
        o = moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)
        dy, dw = moe.moe_unpermute_backward(dout, y, r.perm, r.weights, dy=b)
        return xs, o, dy, dw

    with torch.cuda.stream(stream):
        step(bufs[0], bufs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step(bufs[0], bufs[1])
    for seed in (1, 2, 3):  # new routing and new rows in place
        n = Routed(moe, M, E, k, 16, 10 + seed, drop=0.1)
        r.perm.copy_(n.perm)
        r.weights.copy_(n.weights)
        x.copy_(randn(gen(seed), M, H))
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step(bufs[2], bufs[3])):
            assert torch.equal(a, b)
