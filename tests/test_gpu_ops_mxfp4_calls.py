"""Calls of the 4-bit operators that the documentation allows beside the usual ones:
pre-activations without an activation, one bias of the two, scale bytes that begin anywhere
at every form and depth, and positions past the rows."""

import pytest
import torch

from mx_forms_cases import DEPTHS, FORWARD
from mx_testlib import MX, mx_rows, mx_values, mx_weight, reference
from ops_testlib import assert_within, gen, half, randn, untouched_buffer
from test_gpu_ops_linear import rows_of

pytestmark = pytest.mark.gpu

BF = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def shifted(t, by):
    flat = torch.zeros(t.numel() + 4, dtype=torch.uint8, device="cuda")
    v = flat[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("rows", [5, 300, 1100])
@pytest.mark.parametrize("rows4", [False, True])
@pytest.mark.parametrize("act,first,second", [("none", False, False), ("none", True, False), ("swiglu", True, False), ("swiglu", False, True)])
def test_preact_and_either_bias(moe, rows, rows4, act, first, second):
    N, K, g = 1056, 224, gen(rows)
    r = rows_of(moe, rows, 0)
    x, xs = mx_rows(g, rows, K) if rows4 else (randn(g, rows, K), None)
    w, up = mx_weight(g, 1, N, K), mx_weight(g, 1, N, K) if act == "swiglu" else None
    b, ub = randn(g, 1, N) if first else None, randn(g, 1, N) if second else None
    y, _, pre = moe.moe_grouped_linear_mxfp4(x, w, act=act, up=up, bias=b, up_bias=ub, x_scale=xs, save_preact=True)
    ref, err, pref, perr = reference(r, mx_values(x, xs) if rows4 else x.double(), w, up, b, ub, None, act)
    assert_within(y, ref, BF * (ref.abs() + err) + err + 1e-37, "y")
    assert_within(pre, pref, BF * (pref.abs() + perr) + perr + 1e-37, "preact")
    if act == "none":
        assert torch.equal(y, pre)


@pytest.mark.parametrize("form,rows,N,rows4", [(f, r, n, q) for f, r, n, which in FORWARD for q in (False, True)
                                               if which in ("both", "mxfp4" if q else "bf16")], ids=str)
@pytest.mark.parametrize("K", DEPTHS)
def test_scale_bytes_anywhere(moe, form, rows, N, rows4, K):
    """The bytes' place in memory changes nothing."""
    g, r = gen(N + K), rows_of(moe, rows, N + K)
    x, xs = mx_rows(g, r.rows, K) if rows4 else (randn(g, r.rows, K), None)
    w, up = mx_weight(g, r.E, N, K), mx_weight(g, r.E, N, K)

    def product(by):
        at = (lambda t, i: t) if by == 0 else (lambda t, i: shifted(t, 1 + (by + i) % 3))
        s = None if xs is None else at(xs, 0)
        return moe.moe_grouped_linear_mxfp4(x, (w[0], at(w[1], 1)), r.offsets, r.counts, act="swiglu", up=(up[0], at(up[1], 2)), x_scale=s)[0]

    first = product(0)
    for by in (1, 2, 3):
        assert torch.equal(product(by)[r.kept], first[r.kept]), by


def test_positions_past_the_rows(moe):
    """A slot whose position is not below the rows goes nowhere, as a dropped one."""
    M, H, rows = 6, 96, 4
    x = randn(gen(3), M, H)
    perm = torch.tensor([0, 4, 3, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    codes, scales = untouched_buffer(rows + 2, H // 2, dtype=torch.uint8), untouched_buffer(rows + 2, H // MX, dtype=torch.uint8)
    keep = codes.clone(), scales.clone()
    moe.moe_mxfp4_quantize(x, perm, 1, rows, codes=codes[:rows], scales=scales[:rows])
    plain = moe.moe_mxfp4_quantize(x)
    for got, old, want in zip((codes, scales), keep, plain):
        assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[2])
        assert torch.equal(got[[1, 2, 4, 5]], old[[1, 2, 4, 5]])
