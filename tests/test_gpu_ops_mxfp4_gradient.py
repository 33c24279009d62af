"""The rows' gradient through MXFP4 weights against differences of the products, and the
places that tiles take: a row has the same bits wherever its expert stands among the others,
and when all others are empty."""

import pytest
import torch

from moe_testlib import log
from mx_testlib import mx_values, mx_weight
from ops_testlib import SUM, gen, half, randn

pytestmark = pytest.mark.gpu

BF = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.mark.parametrize("rows,N,K", [(40, 72, 160), (300, 200, 544), (1100, 136, 1056)])
@pytest.mark.parametrize("gated", [False, True])
def test_against_differences(moe, rows, N, K, gated):
    """For every row, <c, W x> moves by <dx, s> over a step s along the gradient itself, so
    that what it moves by is a sum of squares: a gradient of zeros, of another size or
    another sign is far outside.  Bounds: each of the two products is rounded to bf16 and
    summed in float32, as dx is."""
    g = gen(21)
    wide = 2 if gated else 1
    x, c = randn(g, rows, K), randn(g, rows, wide * N)
    weights = [mx_weight(g, 1, N, K) for _ in range(wide)]
    m = torch.cat([mx_values(w[0][0], w[1][0]) for w in weights])
    dx = moe.moe_grouped_linear_mxfp4_backward_x(c, weights[0], up=weights[1] if gated else None).double()
    moved_to = (x.double() + c.double() @ m).bfloat16()
    step = moved_to.double() - x.double()
    moved, bound = 0.0, (BF + (wide * N + 8) * SUM) * ((c.double().abs() @ m.abs()) * step.abs()).sum(1)
    for at, sign in ((moved_to, 1.0), (x, -1.0)):
        y = torch.cat([moe.moe_grouped_linear_mxfp4(at, w)[0] for w in weights], 1).double()
        moved = moved + sign * (y * c.double()).sum(1)
        exact, size = at.double() @ m.T, at.double().abs() @ m.abs().T
        bound = bound + ((BF * exact.abs() + 2 * (K + 8) * SUM * size) * c.double().abs()).sum(1)
    assert bool((moved > 4 * bound).all()), float((moved / bound).min())
    assert bool(((moved - (dx * step).sum(1)).abs() <= bound).all())


def runs(counts):
    offsets = torch.zeros(counts.numel() + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets


# 128 x 128 tiles; 32 x 128, more than run at once; 256 x 256 in the order of their cost
@pytest.mark.parametrize("E,most,N,K", [(24, 300, 672, 672), (128, 50, 544, 288), (16, 1200, 1056, 544)])
@pytest.mark.parametrize("rows4", [False, True])
def test_a_row_has_the_same_bits_in_any_place(moe, E, most, N, K, rows4):
    log(f"places of tiles: {E} experts of up to {most} rows, {N} x {K}, rows4={rows4}")
    g = gen(17)
    counts = torch.randint(0, most, (E,), generator=g, device="cuda", dtype=torch.int32)
    offsets, rows = runs(counts), int(counts.sum())
    order = torch.randperm(E, generator=g, device="cuda")
    moved = runs(counts[order])
    off, cnt, there = offsets.tolist(), counts.tolist(), moved.tolist()
    source = torch.cat([torch.arange(off[e], off[e] + cnt[e], device="cuda") for e in order.tolist()])
    x, dz = randn(g, rows, K), randn(g, rows, 2 * N)
    w, up = mx_weight(g, E, N, K), mx_weight(g, E, N, K)
    w2, up2 = (tuple(t[order].contiguous() for t in v) for v in (w, up))

    def products(rows_in, dz_in, weights, ups, o, c):
        a, s = moe.moe_mxfp4_quantize(rows_in) if rows4 else (rows_in, None)
        y, _, pre = moe.moe_grouped_linear_mxfp4(a, weights, o, c, act="swiglu", up=ups, x_scale=s, save_preact=True)
        return y, pre, moe.moe_grouped_linear_mxfp4_backward_x(dz_in, weights, o, c, up=ups)

    first = products(x, dz, w, up, offsets, counts)
    elsewhere = products(x[source], dz[source], w2, up2, moved, counts[order].contiguous())
    for a, b in zip(first, elsewhere):
        assert torch.equal(a[source], b)
    for e in (int(counts.argmax()), 0, E // 2, E - 1):
        only = torch.zeros_like(counts)
        only[e] = counts[e]
        part = slice(off[e], off[e] + cnt[e])
        for a, b in zip(first, products(x, dz, w, up, offsets, only)):
            assert torch.equal(a[part], b[part]), e
