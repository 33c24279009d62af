"""The norm of rows whose squares, or whose rstd, leave float32's range: every finite
row has the formula's result.

rstd is float32: where (mean z^2 + eps)^(-1/2) is below the smallest normal float it is
rounded to a multiple of 2^-149, and past the largest it is an infinity; y does not
go through it and keeps its precision."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import SUM, assert_within, check_fp8_rows, gen, half

pytestmark = pytest.mark.gpu

DEPTH = 32 + 6 + 16  # of the float32 row sums
TINY = 2.0 ** -133   # half of the smallest bf16 subnormal
MAX = (2 - 2.0 ** -7) * 2.0 ** 127  # the largest bf16


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def rows(H, sizes, g):
    """Rows of +-size times 1, 1/2 or 1/4, the largest value never above bf16's."""
    x = torch.tensor(sizes, dtype=torch.float64, device="cuda")[:, None].repeat(1, H)
    x *= 2.0 ** -torch.randint(0, 3, x.shape, generator=g, device="cuda").double()
    return x * (1 - 2.0 * torch.randint(0, 2, x.shape, generator=g, device="cuda").double())


def check(moe, x, r, z, w, eps):
    fp8 = z.shape[1] % 128 == 0
    y, _, zo, rstd = moe.moe_add_rms_norm(x, w, eps, residual=r, save_rstd=True)
    codes = moe.moe_add_rms_norm(x, w, eps, residual=r, fp8=True) if fp8 else None
    torch.cuda.synchronize()
    if r is not None:
        assert torch.equal(zo.double(), z)
    rr = (z.square().mean(1) + eps) ** -0.5
    rel = (DEPTH / 2 + 8) * SUM
    fits = rr < 2.0 ** 127
    assert_within(rstd[fits], rr[fits], rr[fits] * rel + 2.0 ** -149, "rstd")
    assert bool((rstd[rr >= 2.0 ** 128 * (1 + rel)] == float("inf")).all())
    yr = z * rr[:, None] * w.double()
    assert_within(y, yr, yr.abs() * (half(torch.bfloat16) * (1 + rel) + rel + 2 * SUM) + TINY, "y")
    if fp8:
        check_fp8_rows(codes[0], codes[1], yr, yr.abs() * (rel + 2 * SUM))


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("H", [8, 64, 1000, 1024, 2048, 12000, 32768])
def test_bf16_rows(moe, H, eps):
    log(f"norm range H={H} eps={eps}")
    g = gen(H)
    x = rows(H, [MAX, 2.0 ** 127, 2.0 ** 124, 2.0 ** 121, 2.0 ** 112, 2.0 ** 64, 2.0 ** 50, 2.0 ** -49, 2.0 ** -51, 2.0 ** -70,
                 2.0 ** -100, 2.0 ** -124, 2.0 ** -126, 2.0 ** -131], g).to(torch.bfloat16)
    w = (1 + torch.randint(0, 3, (H,), generator=g, device="cuda") / 4).to(torch.bfloat16)
    check(moe, x, None, x.double(), w, eps)


@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-30])
@pytest.mark.parametrize("H", [8, 1024, 7168, 32768])
def test_float32_rows(moe, H, eps):
    log(f"norm range float32 H={H} eps={eps}")
    g = gen(H + 1)
    z = rows(H, [2.0 ** 127, 2.0 ** 120, 2.0 ** 100, 2.0 ** -52, 2.0 ** -80, 2.0 ** -120, 2.0 ** -126, 2.0 ** -135, 2.0 ** -140,
                 2.0 ** -145], g)
    r = z.float()
    assert torch.equal(r.double(), z)
    w = (1 + torch.randint(0, 3, (H,), generator=g, device="cuda") / 4).to(torch.bfloat16)
    check(moe, torch.zeros(z.shape, dtype=torch.bfloat16, device="cuda"), r, z, w, eps)


def test_infinite_rows_as_before(moe):
    """One infinity among finite values: NaN there, zeros elsewhere."""
    x = torch.ones(2, 2048, dtype=torch.bfloat16, device="cuda")
    x[0, 5] = float("inf")
    x[1] = 2.0 ** 127
    x[1, 9] = float("-inf")
    y, _, _, rstd = moe.moe_add_rms_norm(x, torch.ones(2048, dtype=torch.bfloat16, device="cuda"), 1e-6, save_rstd=True)
    torch.cuda.synchronize()
    assert not bool(rstd.any())
    for m, c in ((0, 5), (1, 9)):
        assert bool(y[m, c].isnan()) and int(y[m].isnan().sum()) == 1 and int((y[m] == 0).sum()) == 2047
