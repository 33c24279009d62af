"""The products at the largest row counts the library takes, just below 2^31 (8 columns:
34 GB a matrix): every row is computed, and none past the end is read."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import SUM, gen, half, randn

pytestmark = pytest.mark.gpu

MOST, C, TAIL = 2 ** 31 - 1, 8, 700
BF = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.fixture(scope="module")
def x():
    free, _ = torch.cuda.mem_get_info()
    if free < 120e9:
        pytest.skip("needs 120 GB of GPU memory")
    t = torch.ones(MOST, C, dtype=torch.bfloat16, device="cuda")
    t[:TAIL] = randn(gen(1), TAIL, C)
    t[-TAIL:] = randn(gen(2), TAIL, C)
    yield t
    del t
    torch.cuda.empty_cache()


def ends():
    return slice(0, TAIL), slice(MOST - TAIL, MOST)


def assert_rows(got, ref, mag, what):
    """got (bf16, [MOST, C]) against ref(part) in float64 at both ends, and everywhere
    between the row of ones' value."""
    for part in ends():
        r, m = ref(part), mag(part)
        assert bool(((got[part].double() - r).abs() <= BF * r.abs() + 16 * SUM * m).all()), (what, part)
    step = 1 << 27
    one = got[TAIL].clone()
    for at in range(TAIL, MOST - TAIL, step):
        assert bool((got[at:min(at + step, MOST - TAIL)] == one).all()), (what, at)


@pytest.mark.parametrize("grouped", [False, True])
def test_product_and_rows_gradient(moe, x, grouped):
    log(f"products of {MOST} rows, grouped={grouped}")
    w = randn(gen(3), 1, C, C)
    runs = ()
    if grouped:
        runs = (torch.tensor([0, MOST], dtype=torch.int32, device="cuda"), torch.tensor([MOST], dtype=torch.int32, device="cuda"))
    out = torch.full((MOST, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear(x, w, *runs, out=out)
    torch.cuda.synchronize()
    assert_rows(out, lambda p: x[p].double() @ w[0].double().T, lambda p: x[p].double().abs() @ w[0].double().abs().T, "y")
    log("rows' gradient")
    out.fill_(float("nan"))
    moe.moe_grouped_linear_backward_x(x, w, *runs, dx=out)
    torch.cuda.synchronize()
    assert_rows(out, lambda p: x[p].double() @ w[0].double(), lambda p: x[p].double().abs() @ w[0].double().abs(), "dx")


def test_activation_gradient(moe, x):
    log(f"activation gradient of {MOST} rows")
    out = torch.full((MOST, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_act_backward(x, x, "silu", dz=out)
    torch.cuda.synchronize()

    def ref(p):
        z = x[p].double()
        s = torch.sigmoid(z)
        return z * s * (1 + z * (1 - s))

    assert_rows(out, ref, lambda p: 2 * x[p].double().abs(), "dz")


@pytest.mark.parametrize("cut", [8000, 7])  # in the first the last row split begins where 31 bits end
def test_weight_gradient(moe, x, cut):
    rows = MOST - cut
    log(f"weights' gradient of {rows} rows")
    dz = torch.zeros(MOST, C, dtype=torch.bfloat16, device="cuda")
    dz[rows:] = float("nan")  # past the end of what the call is given
    at = torch.tensor([0, 1, 4194303, 4194304, 2 ** 30, rows - 4194305, rows - 2, rows - 1], device="cuda")
    dz[at] = randn(gen(5), len(at), C)
    dw, _, db, _ = moe.moe_grouped_linear_backward_w(dz[:rows], x[:rows], bias=True, dtype=torch.float32)
    torch.cuda.synchronize()
    d, xx = dz[at].double(), x[at].double()
    assert bool(((dw[0].double() - d.T @ xx).abs() <= 32 * SUM * (d.abs().T @ xx.abs())).all())
    assert bool(((db[0].double() - d.sum(0)).abs() <= 32 * SUM * d.abs().sum(0)).all())
