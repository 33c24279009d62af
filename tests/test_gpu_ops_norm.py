"""The RMS norm with the residual's addition and its gradient against the
formulas in float64 (bounds: see ops_testlib)."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import SUM, assert_within, check_fp8_rows, gen, half, randn

pytestmark = pytest.mark.gpu

EPS = 1e-6
TINY = 2.0 ** -133  # half of the smallest bf16 subnormal
# depth of the float32 row sums: at most 32 elements a thread, then waves and wave parts
DEPTH = 32 + 6 + 16


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def inputs(M, H, seed, res):
    g = gen(seed)
    x = randn(g, M, H)
    w = randn(g, H, scale=0.2) + 1.0
    r = None if res is None else randn(g, M, H, scale=3.0, dtype=res)
    return x, w, r


def reference(x, w, r):
    z = x.double()
    if r is not None:
        # the float32 sum of two bf16 values rounded to the residual's type
        z = (x.float() + r.float()).to(r.dtype).double()
    rstd = (z.square().mean(1) + EPS) ** -0.5
    return z, rstd, z * rstd[:, None] * w.double()


SHAPES = [(1, 2048), (3, 1), (5, 7), (2, 64), (4, 513), (7, 2048), (2, 2049), (3, 4096), (2, 7168), (2, 8191), (3, 12000),
          (2, 32768), (2500, 264), (2300, 1000), (2200, 2047), (1, 16384)]


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", SHAPES)
def test_forward(moe, M, H, res):
    log(f"norm M={M} H={H} residual={res}")
    x, w, r = inputs(M, H, M * 7 + H, res)
    y, scale, z, rstd = moe.moe_add_rms_norm(x, w, EPS, residual=r, save_rstd=True)
    torch.cuda.synchronize()
    assert scale is None and (z is None) == (r is None)
    zr, rr, yr = reference(x, w, r)
    if r is not None:
        assert torch.equal(z.double(), zr)
    # rstd: half the relative error of the mean, plus division, root and reciprocal
    rel = (DEPTH / 2 + 4) * SUM
    assert_within(rstd, rr, rr * rel, "rstd")
    assert_within(y, yr, yr.abs() * (half(torch.bfloat16) * (1 + rel) + rel + 2 * SUM) + TINY, "y")


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", [(1, 128), (3, 384), (5, 2048), (2, 7168), (2100, 640), (2, 16384), (2, 32768)])
def test_forward_8bit(moe, M, H, res):
    log(f"norm 8-bit M={M} H={H} residual={res}")
    x, w, r = inputs(M, H, M + H, res)
    x[0, :128] = 0
    if r is not None:
        r[0, :128] = 0  # a block of zeros: scale 1
    codes, scale, _, _ = moe.moe_add_rms_norm(x, w, EPS, residual=r, fp8=True)
    torch.cuda.synchronize()
    _, _, yr = reference(x, w, r)
    check_fp8_rows(codes, scale, yr, yr.abs() * ((DEPTH / 2 + 6) * SUM))
    assert float(scale[0, 0]) == 1.0 and not bool(codes[0, :128].float().any())


def test_extreme_rows(moe):
    """A row of zeros, the smallest and the largest values, a NaN and an infinity."""
    H = 256
    x = torch.ones(6, H, dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1] = 2.0 ** -70           # squares underflow: eps alone is left
    x[2] = 2.0 ** 60
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, _, _, _ = moe.moe_add_rms_norm(x, w, EPS)
    codes, scale, _, _ = moe.moe_add_rms_norm(x, w, EPS, fp8=True)
    torch.cuda.synchronize()
    assert not bool(y[0].float().any()) and bool((scale[0] == 1).all())
    assert_within(y[1], torch.full((H,), 2.0 ** -70 * EPS ** -0.5, device="cuda"), 2.0 ** -70 * EPS ** -0.5 * 2.0 ** -7)
    assert_within(y[2], torch.ones(H, device="cuda"), 2.0 ** -7)
    assert bool(y[3].isnan().all()) and bool(scale[3].isnan().all())
    # an infinite mean: the infinity itself becomes NaN, the finite values 0
    assert bool(y[4, 7].isnan()) and int(y[4].isnan().sum()) == 1
    assert bool(scale[4, 0].isnan()) and float(scale[4, 1]) == 1.0
    assert bool(codes[4].float()[:128].isnan().all()) and not bool(codes[4, 128:].float().any())
    assert bool((y[5] == 1).all())


def test_strides_in_place_and_alignment(moe):
    """x as a column slice of a wider matrix at an odd element offset, the stream
    updated in place, and the same bits as from fresh contiguous buffers."""
    for M, H in ((6, 1000), (2100, 520)):
        g = gen(H)
        wide = randn(g, M, H + 37)
        x = wide[:, 3:3 + H]
        w = randn(g, H) + 1.0
        r = randn(g, M, H)
        y0, _, z0, _ = moe.moe_add_rms_norm(x.contiguous(), w, EPS, residual=r)
        y1, _, z1, _ = moe.moe_add_rms_norm(x, w, EPS, residual=r, residual_out=r)
        assert z1.data_ptr() == r.data_ptr()
        assert torch.equal(y0, y1) and torch.equal(z0, r)
        xc = x.contiguous()
        y2, _, _, _ = moe.moe_add_rms_norm(xc, w, EPS)
        y3, _, _, _ = moe.moe_add_rms_norm(xc, w, EPS, out=xc)  # over its own input
        assert torch.equal(y2, y3)


def test_rows_are_independent(moe):
    x, w, r = inputs(40, 2048, 3, torch.bfloat16)
    y, _, _, rstd = moe.moe_add_rms_norm(x, w, EPS, residual=r, save_rstd=True)
    for m in (1, 2, 5):
        a, _, _, b = moe.moe_add_rms_norm(x[:m].contiguous(), w, EPS, residual=r[:m].contiguous(), save_rstd=True)
        assert torch.equal(a, y[:m]) and torch.equal(b, rstd[:m])


@pytest.mark.parametrize("zt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_dz", [True, False])
@pytest.mark.parametrize("M,H", [(1, 2048), (3, 1), (5, 7), (9, 513), (300, 2048), (33, 4096), (17, 7168), (3, 12000), (2, 32768),
                                 (9000, 264), (5000, 1000)])
def test_backward(moe, M, H, zt, with_dz):
    log(f"norm backward M={M} H={H} {zt} dz={with_dz}")
    g = gen(M + H)
    z = randn(g, M, H, scale=2.0, dtype=zt)
    w = randn(g, H, scale=0.2) + 1.0
    dy = randn(g, M, H)
    dz = randn(g, M, H, dtype=zt) if with_dz else None
    rstd = (z.double().square().mean(1) + EPS).pow(-0.5).float()
    dx, dw = moe.moe_add_rms_norm_backward(dy, z, w, rstd, dz=dz)
    torch.cuda.synchronize()
    r = rstd.double()[:, None]
    n = z.double() * r
    t = dy.double() * w.double()
    dot = (t * n).mean(1, keepdim=True)
    ref = r * (t - n * dot) + (dz.double() if with_dz else 0.0)
    mag = r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True)) + (dz.double().abs() if with_dz else 0.0)
    assert_within(dx, ref, half(zt) * ref.abs() + (DEPTH + 8) * SUM * mag + 1e-37, "dx")
    assert_within(dw, (dy.double() * n).sum(0), (M + 16) * SUM * (dy.double() * n).abs().sum(0) + 1e-37, "dw")
    if zt == torch.bfloat16:  # over the buffer of dy
        own = dy.clone()
        again, dw2 = moe.moe_add_rms_norm_backward(own, z, w, rstd, dz=dz, dx=own)
        assert torch.equal(again, dx) and torch.equal(dw2, dw)
    # without the weight's gradient, and over the buffer of dz
    again, none = moe.moe_add_rms_norm_backward(dy, z, w, rstd, dz=dz, need_dweight=False, dx=dz)
    assert none is None and torch.equal(again, dx)


def test_backward_is_the_derivative(moe):
    """The gradient against central differences of the formula in float64."""
    M, H = 3, 48
    g = gen(11)
    z, w, dy = randn(g, M, H, dtype=torch.float32), randn(g, H) + 1.0, randn(g, M, H)

    def f(zz, ww):
        return (zz * (zz.square().mean(1, keepdim=True) + EPS).pow(-0.5) * ww * dy.double()).sum()

    rstd = (z.double().square().mean(1) + EPS).pow(-0.5).float()
    dx, dw = moe.moe_add_rms_norm_backward(dy, z, w, rstd)
    h = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 47)):
        d = torch.zeros(M, H, dtype=torch.float64, device="cuda")
        d[i, j] = h
        num = (f(z.double() + d, w.double()) - f(z.double() - d, w.double())) / (2 * h)
        assert abs(float(num) - float(dx[i, j])) <= 1e-5
        num = (f(z.double(), w.double() + d[i]) - f(z.double(), w.double() - d[i])) / (2 * h)
        assert abs(float(num) - float(dw[j])) <= 1e-4


def test_no_rows(moe):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, _, _, _ = moe.moe_add_rms_norm(x, w, EPS)
    assert y.shape == (0, 256)
    dx, dw = moe.moe_add_rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and not bool(dw.any())


def test_graph_replay_and_stream(moe):
    """Captured forward and backward replay for new inputs, also with eager calls between."""
    M, H = 600, 2048
    x, w, r = inputs(M, H, 5, torch.bfloat16)
    dy = randn(gen(6), M, H)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        y, _, z, rstd = moe.moe_add_rms_norm(x, w, EPS, residual=r, save_rstd=True)
        dx, dw = moe.moe_add_rms_norm_backward(dy, z, w, rstd, dz=z)
        return y, z, rstd, dx, dw

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    for seed in (1, 2, 3):
        g = gen(seed)
        x.copy_(randn(g, M, H))
        r.copy_(randn(g, M, H))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    # an explicit stream: outputs are allocated on it
    y, _, _, _ = moe.moe_add_rms_norm(x, w, EPS, residual=r, stream=stream)
    stream.synchronize()
    assert torch.equal(y, got[0])


@pytest.mark.parametrize("H", [256, 2048, 12000])
def test_range_of_squares(moe, H):
    """Rows whose squares leave float32's range, with and without eps."""
    x = torch.ones(4, H, dtype=torch.float64, device="cuda")
    x *= torch.tensor([2.0 ** 62, 2.0 ** 120, 2.0 ** -75, 2.0 ** -110], dtype=torch.float64, device="cuda")[:, None]
    x *= 1 + torch.arange(H, device="cuda") % 3
    xb = x.to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    for eps in (0.0, 1e-6):
        y, _, _, rstd = moe.moe_add_rms_norm(xb, w, eps, save_rstd=True)
        torch.cuda.synchronize()
        z = xb.double()
        rr = (z.square().mean(1) + eps) ** -0.5
        rel = (DEPTH / 2 + 8) * SUM
        assert_within(rstd, rr, rr * rel + 2.0 ** -149, "rstd")
        yr = z * rr[:, None]
        # rstd near 2^-121 is a normal float; 2^-128 of rounding below that is counted
        assert_within(y, yr, yr.abs() * (half(torch.bfloat16) * (1 + rel) + rel + 2 * SUM) + TINY, "y")
