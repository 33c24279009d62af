"""Gradients clipped at the ends of float32's range: factors below its smallest normal
number, and norms past its largest one.

A clipped value is g * max_norm / norm with the norm rounded to float32: one rounding of
the norm (relative, half of float32's), one of the result to float32, and one to its type;
below the smallest normal number a rounding is off by half of the smallest subnormal.  The
steps in 64 bits between them add less than 2^-50."""

import math

import pytest
import torch

from moe_testlib import log
from ops_testlib import assert_within, gen, half

pytestmark = pytest.mark.gpu

F32 = half(torch.float32)
BF16, FP32 = torch.bfloat16, torch.float32
SUBNORMAL = {FP32: 2.0 ** -150, BF16: 2.0 ** -134}  # half of the smallest one


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def randoms(scale, types, sizes=(9000, 5, 0, 20000)):
    return [(torch.randn(n, generator=gen(n + 1), device="cuda") * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def assert_scaled(out, before, factor):
    for o, b in zip(out, before):
        ref = b.double() * factor
        bound = ref.abs() * (2 * F32 + 2.0 ** -50) + SUBNORMAL[FP32]
        if b.dtype == BF16:
            bound = bound + (ref.abs() + bound) * half(BF16) + SUBNORMAL[BF16]
        assert_within(o, ref, bound)


# norms of about 1.7e2, 1.7e38 and 1.7e-37, by factors down to 2^-146, below which nothing is left
@pytest.mark.parametrize("types", [(FP32,), (BF16,), (FP32, BF16)], ids=str)
@pytest.mark.parametrize("scale,max_norm", [(1e36, 1.0), (1e36, 1e-4), (1e36, 3e-7), (1.0, 1e-36), (1.0, 1e-41), (1e-39, 1e-42)])
def test_small_factors(moe, types, scale, max_norm):
    log(f"clip {types} scale={scale} max_norm={max_norm}")
    grads = randoms(scale, types)
    before = [g.clone() for g in grads]
    norm = moe.moe_grad_norm(grads)
    want = min(1.0, float(torch.tensor(max_norm)) / norm64(grads))
    out = [torch.full_like(g, 7.0) for g in grads]
    assert torch.equal(moe.moe_clip_grad_norm(grads, max_norm, out=out), norm)
    assert_scaled(out, before, want)
    two = [torch.empty_like(g) for g in grads]
    moe.moe_grad_clip(grads, norm, max_norm, out=two)
    assert all(torch.equal(a, b) for a, b in zip(out, two))
    moe.moe_clip_grad_norm(grads, max_norm)  # in place
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


def test_no_norm_at_all(moe):
    """A largest norm of zero makes zeros of everything finite."""
    grads = randoms(1e30, (FP32, BF16))
    moe.moe_clip_grad_norm(grads, 0.0)
    assert not any(bool(g.any()) for g in grads)


@pytest.mark.parametrize("types", [(FP32,), (BF16,), (FP32, BF16)], ids=str)
@pytest.mark.parametrize("max_norm", [1.0, 1e30, 3e38, 1e-10])
def test_norm_past_float32(moe, types, max_norm):
    """Finite gradients whose norm (about 5e39) float32 cannot hold are clipped by it all the
    same; the norm that is returned is an infinity, by which moe_grad_clip scales nothing."""
    log(f"clip {types} past float32, max_norm={max_norm}")
    grads = randoms(3e37, types)
    before = [g.clone() for g in grads]
    assert all(bool(g.isfinite().all()) for g in grads) and norm64(grads) > 3.5e38
    want = float(torch.tensor(max_norm)) / norm64(grads)
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = moe.moe_clip_grad_norm(grads, max_norm, out=out)
    assert bool(norm.isinf())
    assert_scaled(out, before, want)
    apart = [torch.full_like(g, 7.0) for g in grads]
    assert bool(moe.moe_grad_norm(grads).isinf())
    moe.moe_grad_clip(grads, norm, max_norm, out=apart)
    assert all(torch.equal(a, b) for a, b in zip(apart, before))
    assert bool(moe.moe_clip_grad_norm(grads, max_norm).isinf())  # in place
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_beside_large_ones(moe, value):
    """A gradient that is not finite still scales nothing, however large the others are."""
    grads = randoms(3e37, (FP32,))
    grads[0][17] = value
    before = [g.clone() for g in grads]
    norm = moe.moe_clip_grad_norm(grads, 1.0)
    assert bool(norm.isnan() if value != value else norm == float("inf"))
    for g, b in zip(grads, before):
        assert torch.equal(g.nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0))


def test_nothing_to_clip_writes_nothing_in_place(moe):
    """Where nothing is scaled, a gradient that is clipped in place keeps its very bits,
    beside others that are copied: a signalling NaN would come back as a quiet one."""
    signalling = 0x7F81  # bf16
    there = torch.full((9000,), signalling, dtype=torch.int16, device="cuda").view(BF16)
    wide = torch.full((3000,), signalling << 16, dtype=torch.int32, device="cuda").view(FP32)
    other = torch.ones(9000, device="cuda")
    copy = torch.zeros_like(other)
    for call in (lambda: moe.moe_clip_grad_norm([there, other, wide], 1.0, out=[there, copy, wide]),
                 lambda: moe.moe_grad_clip([there, other, wide], torch.tensor([1.0], device="cuda"), 1.0, out=[there, copy, wide])):
        copy.zero_()
        call()
        assert torch.equal(copy, other)
        assert bool((there.view(torch.int16) == signalling).all()) and bool((wide.view(torch.int32) == signalling << 16).all())
