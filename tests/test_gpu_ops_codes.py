"""8-bit rows bit for bit: a block's scale is its absolute maximum over 448 and its
codes are e4m3fn(y / scale), the quotient rounded to float32 once (no tolerance: the
float32 y that is divided is known exactly in these cases, and bf16 inputs put many
quotients on the border between two codes, where any other rounding shows)."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import BLOCK, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def over(a, b):
    """a / b rounded to float32 once: the float64 quotient of float32 values has bits
    enough that rounding it again changes nothing.  (torch divides by a number on the
    GPU by multiplying with its rounded reciprocal.)"""
    return (a.double() / b).float()


def assert_same_rows(codes, scale, y, what):
    b = y.reshape(y.shape[0], -1, BLOCK)
    amax = b.abs().amax(2)
    ws = torch.where(amax > 0, over(amax, 448.0).clamp(min=2.0 ** -126), torch.ones_like(amax))
    want = over(b, ws.double()[..., None]).reshape(y.shape).to(torch.float8_e4m3fn)
    assert torch.equal(scale, ws), (what, "scale", int((scale != ws).sum()))
    off = codes.view(torch.uint8) != want.view(torch.uint8)
    assert not bool(off.any()), (what, "codes", int(off.sum()), off.numel())


@pytest.mark.parametrize("M,H", [(4096, 512), (3000, 1024), (700, 2048), (300, 7168), (64, 16384), (16, 32768)])
@pytest.mark.parametrize("exp", [0, 90, -58, -66, -110, -124])  # scales down to the smallest, 2^-126
def test_norm_codes(moe, M, H, exp):
    log(f"norm codes M={M} H={H} weights around 2^{exp}")
    g = gen(M + H)
    x, w = randn(g, M, H), randn(g, H, scale=0.2) + 1.0
    x[0, 3] = 0.0
    x[0, 4] = -0.0
    w = (w.double() * 2.0 ** exp).to(torch.bfloat16)
    codes, scale, _, rstd = moe.moe_add_rms_norm(x, w, 1e-6, fp8=True, save_rstd=True)
    torch.cuda.synchronize()
    # y = (z * rstd) * weight, two float32 products in this order
    assert_same_rows(codes, scale, x.float() * rstd[:, None] * w.float(), "norm")


def identity(E, N, copies):
    """[E, N, copies * N]: row n sums the elements n, N + n, ... of x."""
    return torch.eye(N, dtype=torch.bfloat16, device="cuda").repeat(1, copies).expand(E, -1, -1).contiguous()


# rows of one dense product by the form they take: depth-split, 128 x 128, 256 x 256
# tiles (bf16 operands; 8-bit operands take 128 x 128 for both)
@pytest.mark.parametrize("rows,N", [(20, 512), (1000, 512), (4100, 4224)])
@pytest.mark.parametrize("fp8", [False, True])
def test_product_codes(moe, rows, N, fp8):
    log(f"product codes rows={rows} N={N} fp8={fp8}")
    g = gen(rows + N + fp8)
    if fp8:  # y = code * scale, exact in float32 for a power of two
        x = (torch.randn(rows, N, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)  # below 448
        xs = 2.0 ** torch.randint(-3, 4, (rows, N // BLOCK), generator=g, device="cuda").float()
        eye = identity(1, N, 1).to(torch.float8_e4m3fn).view(torch.uint8)
        w = (eye, torch.ones(1, N // BLOCK, N // BLOCK, device="cuda"))
        codes, scale, _ = moe.moe_grouped_linear(x, w, x_scale=xs, fp8_out=True)
        y = x.float() * xs.repeat_interleave(BLOCK, 1) + 0.0  # the sum's zeros: -0 becomes 0
    else:  # y = hi + lo, 16 bits of two bf16 columns
        hi = randn(g, rows, N)
        lo = torch.where(torch.rand(rows, N, generator=g, device="cuda") < 0.5, hi * 2.0 ** -9, 0.0).to(torch.bfloat16)
        codes, scale, _ = moe.moe_grouped_linear(torch.cat([hi, lo], 1), identity(1, N, 2), fp8_out=True)
        y = hi.float() + lo.float()
    torch.cuda.synchronize()
    assert_same_rows(codes, scale, y, "product")
    # the residual is added in float32 before the rounding
    if not fp8:
        r = randn(g, rows, N, scale=2.0 ** -8)
        codes, scale, _ = moe.moe_grouped_linear(torch.cat([hi, lo], 1), identity(1, N, 2), residual=r, fp8_out=True)
        torch.cuda.synchronize()
        assert_same_rows(codes, scale, (hi.float() + lo.float()) + r.float(), "product + residual")


def near_midpoints():
    """Pairs (v, s) of 24-bit integers whose quotient is |d| <= 3 units of 1 / s from the
    middle of two floats, of which one is the border t of two codes: v 2^k = M s + d for
    M = t 2^20 +- 1, a float and a half in units of half a step."""
    for t in range(17, 32, 2):
        for m in (t * 2 ** 20 + 1, t * 2 ** 20 - 1):
            for k in range(20, 27):
                for d in (1, -1, 2, -2, 3, -3):
                    v = d * pow(2 ** k, -1, m) % m
                    while v < 2 ** 24:
                        s = (v * 2 ** k - d) // m
                        if v >= 2 ** 23 and 2 ** 23 <= s < 2 ** 24:
                            yield v * 2.0 ** (k - 44), s * 2.0 ** -24
                        v += m


def test_quotients_beside_a_border(moe):
    """Scales and values of 24 bits: the quotients that any error of the division would
    turn to the other code."""
    rows = []
    for v, s in near_midpoints():
        top = torch.tensor(448 * s, dtype=torch.float64).float()
        for amax in (top, torch.nextafter(top, top * 0), torch.nextafter(top, top * 2)):
            if float((amax.double() / 448).float()) == s:
                rows.append([float(amax)] + [(-1) ** c * v * 2.0 ** -(c % 8) for c in range(127)])
                break
    assert len(rows) > 20
    y = torch.tensor(rows, dtype=torch.float64, device="cuda")
    assert torch.equal(y.float().double(), y)
    hi = y.to(torch.bfloat16)
    mid = (y - hi.double()).to(torch.bfloat16)
    lo = (y - hi.double() - mid.double()).to(torch.bfloat16)
    assert torch.equal(hi.double() + mid.double() + lo.double(), y)
    x = torch.cat([hi, mid, lo], 1)  # any sum of the three parts is exact
    for n in (20, len(rows)):
        many = x[:n] if n == 20 else x.repeat(8, 1)
        codes, scale, _ = moe.moe_grouped_linear(many, identity(1, BLOCK, 3), fp8_out=True)
        torch.cuda.synchronize()
        assert_same_rows(codes, scale, y.float()[:n] if n == 20 else y.float().repeat(8, 1), n)
