"""The norm of many gradients together and the gradients clipped by it, against the
formula in float64.

The sums are in 64 bits, so the norm is off by its rounding to float32; the factor
max_norm / norm by two roundings (the norm's and the quotient's), a clipped value by one
more in float32 and one to its type."""

import math

import pytest
import torch

from moe_testlib import log
from ops_testlib import assert_within, gen, half

pytestmark = pytest.mark.gpu

F32 = half(torch.float32)
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(moe, grads, max_norm):
    before = [g.clone() for g in grads]
    want = norm64(grads)
    norm = moe.moe_grad_norm(grads)
    assert norm.shape == (1,) and norm.dtype == FP32
    assert abs(float(norm) - want) <= want * (F32 + 1e-12) + 2.0 ** -150
    out = [torch.full_like(g, 7.0) for g in grads]
    assert torch.equal(moe.moe_clip_grad_norm(grads, max_norm, out=out), norm)
    for g, b, o in zip(grads, before, out):
        assert torch.equal(g, b)  # the gradients themselves stay
        c = min(1.0, max_norm / want) if want > 0 else 1.0
        ref = b.double() * c
        bound = ref.abs() * 4 * F32 + 2.0 ** -149 if c < 1 else torch.zeros_like(ref)
        if b.dtype == BF16 and c < 1:
            bound = bound + (ref.abs() + bound) * half(BF16) + 2.0 ** -134
        assert_within(o, ref, bound)
    two = [torch.empty_like(g) for g in grads]
    assert moe.moe_grad_clip(grads, norm, max_norm, out=two) == two
    assert all(torch.equal(a, b) for a, b in zip(out, two))
    assert torch.equal(moe.moe_clip_grad_norm(grads, max_norm), norm)  # in place
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


SIZES = [[1], [5], [8192], [8193, 1, 0, 77], [0, 3, 0], [100000, 8191, 16384, 24577], [3] * 300, [9000] * 97, [2_000_001, 1_500_000, 64]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("types", [(BF16,), (FP32,), (BF16, FP32)], ids=str)
@pytest.mark.parametrize("clip", [False, True])
def test_norm_and_clip(moe, sizes, types, clip):
    log(f"clip {len(sizes)} tensors of {sizes[:4]} {types} clip={clip}")
    g = gen(sum(sizes) + len(sizes))
    grads = [(torch.randn(n, generator=g, device="cuda") * (1 + i % 3)).to(types[i % len(types)]) for i, n in enumerate(sizes)]
    want = norm64(grads)
    check(moe, grads, want / 3 if clip else want * 3 + 1)


def test_slices_at_any_element(moe):
    """Gradients that lie in one buffer, begin anywhere in it and have several dimensions."""
    g = gen(3)
    for t in (BF16, FP32):
        pool = torch.randn(60001, generator=g, device="cuda").to(t)
        grads = [pool[1:13].view(3, 4), pool[13:8210], pool[8211:8211 + 70 * 611].view(70, 1, 611), pool[60000:]]
        keep = pool.clone()
        check(moe, grads, 1.5)
        outside = torch.ones_like(pool, dtype=torch.bool)
        for a, b in ((1, 8210), (8211, 8211 + 70 * 611), (60000, 60001)):
            outside[a:b] = False
        assert torch.equal(pool[outside], keep[outside])  # what lies between is untouched


@pytest.mark.parametrize("dtype,scale", [(FP32, 1e30), (FP32, 1e-30), (BF16, 1e30), (BF16, 1e-30)], ids=str)
def test_squares_past_float32(moe, dtype, scale):
    """Squares that overflow or underflow float32 still make the norm."""
    grads = [(torch.randn(5000, generator=gen(4), device="cuda") * scale).to(dtype)]
    check(moe, grads, norm64(grads) / 2)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(moe, value):
    """A norm that is not finite is returned, and the gradients stay as they are."""
    grads = [torch.ones(9000, device="cuda"), torch.ones(300, dtype=BF16, device="cuda")]
    grads[1][7] = value
    before = [g.clone() for g in grads]
    norm = moe.moe_clip_grad_norm(grads, 1.0)
    assert bool(norm.isnan() if value != value else norm == float("inf"))
    out = [torch.zeros_like(g) for g in grads]
    moe.moe_clip_grad_norm(grads, 1.0, out=out)
    for g, b, o in zip(grads, before, out):
        assert torch.equal(g.nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0)) and torch.equal(o.nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0))


def test_borders(moe):
    """Zero gradients, a largest norm of zero, and a norm right at the limit."""
    zero = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(moe.moe_clip_grad_norm(zero, 1.0)) == 0.0 and not bool(zero[0].any())
    assert float(moe.moe_clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    g = [torch.full((4,), 2.0, device="cuda")]  # norm 4
    moe.moe_clip_grad_norm(g, 4.0)
    assert torch.equal(g[0], torch.full((4,), 2.0, device="cuda"))
    moe.moe_clip_grad_norm(g, 0.0)
    assert torch.equal(g[0], torch.zeros(4, device="cuda"))


def test_norm_from_elsewhere(moe):
    """moe_grad_clip takes the norm of more than this process's gradients."""
    g = [torch.ones(10, device="cuda"), torch.full((3,), 2.0, dtype=BF16, device="cuda")]
    moe.moe_grad_clip(g, torch.tensor([8.0], device="cuda"), 2.0)
    assert torch.equal(g[0], torch.full((10,), 0.25, device="cuda")) and torch.equal(g[1], torch.full((3,), 0.5, dtype=BF16, device="cuda"))


def test_same_bits_every_time(moe):
    grads = [torch.randn(3_000_000, generator=gen(9), device="cuda"), torch.randn(70_001, generator=gen(8), device="cuda").bfloat16()]
    norms = {float(moe.moe_grad_norm(grads)) for _ in range(10)}
    assert len(norms) == 1


def test_graph_and_streams(moe):
    """A captured call replays on new gradients; two streams share nothing."""
    grads = [torch.randn(200_000, generator=gen(1), device="cuda"), torch.randn(999, generator=gen(2), device="cuda").bfloat16()]
    out = [torch.empty_like(g) for g in grads]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        moe.moe_clip_grad_norm(grads, 2.0, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        norm = moe.moe_clip_grad_norm(grads, 2.0, out=out)
    for seed in (5, 6, 7):
        for g in grads:
            g.copy_(torch.randn(g.shape, generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got, n = [o.clone() for o in out], norm.clone()
        other = [torch.empty_like(g) for g in grads]
        assert torch.equal(moe.moe_clip_grad_norm(grads, 2.0, out=other), n)
        assert all(torch.equal(a, b) for a, b in zip(got, other))
    sets = [[torch.randn(500_000 + i, generator=gen(i), device="cuda")] for i in (1, 2)]
    want = [moe.moe_grad_norm(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(moe.moe_grad_norm(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals(moe):
    a, b = torch.ones(8, device="cuda"), torch.ones(8, dtype=BF16, device="cuda")
    norm = torch.ones(1, device="cuda")
    for call in (lambda: moe.moe_grad_norm([]), lambda: moe.moe_grad_norm(a), lambda: moe.moe_grad_norm([a.double()]),
                 lambda: moe.moe_grad_norm([a[::2]]), lambda: moe.moe_grad_norm([a, a.cpu()]),
                 lambda: moe.moe_clip_grad_norm([a], -1.0), lambda: moe.moe_clip_grad_norm([a], float("nan")),
                 lambda: moe.moe_clip_grad_norm([a], float("inf")), lambda: moe.moe_clip_grad_norm([a, a], 1.0),
                 lambda: moe.moe_clip_grad_norm([a, b], 1.0, out=[a]), lambda: moe.moe_clip_grad_norm([a], 1.0, out=[b]),
                 lambda: moe.moe_clip_grad_norm([a[:4], a[4:]], 1.0, out=[a[4:], a[:4]]),
                 lambda: moe.moe_grad_clip([a], norm.double(), 1.0)):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
    assert torch.equal(a, torch.ones(8, device="cuda"))
