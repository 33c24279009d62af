"""MXFP4 rows and weights: rounding and reading them back bit for bit, the experts'
products on them and the rows' gradient against the formulas in float64."""

import numpy as np
import pytest
import torch

import oracle
from moe_testlib import log
from mx_testlib import (MX, check_mx_rows, mx_quantised, mx_rows, mx_values, mx_weight, reference, unsigned_zeros)
from ops_testlib import SUM, assert_untouched, assert_within, gen, half, poison, randn, untouched_buffer
from test_gpu_ops_linear import EPILOGUES, ROWS, rows_of

pytestmark = pytest.mark.gpu

BF = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


# ---------------------------------------------------------------- rounding --

def special_rows(dtype):
    """Rows of 64: every border between codes at several scales, the largest and smallest
    values, blocks of zeros, NaN and infinities."""
    ties = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, 0.24, 0.26, 5.03125], device="cuda")
    rows = []
    for e in (-126, -120, -60, -3, 0, 1, 40, 125):
        b = torch.cat([ties, -ties]).double() * 2.0 ** e
        rows.append(torch.cat([b, b / 2]))
    tiny, huge = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    line = torch.linspace(-1, 1, 64, dtype=torch.float64, device="cuda")
    rows += [line * tiny, line * tiny * 2, line * tiny * 5, line * huge, line * 0, line * tiny / 64]
    v = torch.stack(rows).to(dtype)
    bad = torch.stack([line, line, line, line * 0]).to(dtype)
    bad[0, 3], bad[1, 40], bad[2, 63], bad[3, 31] = float("nan"), float("inf"), -float("inf"), float("nan")
    return torch.cat([v, bad])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_special_values(moe, dtype):
    x = special_rows(dtype)
    codes, scales = moe.moe_mxfp4_quantize(x)
    want, bytes_ = mx_quantised(x)
    assert torch.equal(scales, bytes_)
    assert torch.equal(unsigned_zeros(codes), want)
    for dt in (torch.bfloat16, torch.float32):
        got = moe.moe_mxfp4_dequantize(codes, scales, dtype=dt)
        assert got.dtype == dt and torch.equal(got.double().nan_to_num(nan=3.0e38), mx_values(codes, scales).nan_to_num(nan=3.0e38))
    finite = (scales != 255).all(1)
    assert np.array_equal(oracle.mxfp4_decode(codes[finite].cpu().numpy(), scales[finite].cpu().numpy()),
                          mx_values(codes, scales)[finite].cpu().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_every_scale(moe, dtype):
    """All 256 scale bytes with all 16 codes: 2^-128 is the smallest value, exact in either
    type; what passes the largest one is an infinity."""
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None]
    pair = torch.arange(16, dtype=torch.uint8, device="cuda")
    codes = (pair | pair.flip(0) << 4).repeat(256, 1)
    got = moe.moe_mxfp4_dequantize(codes, scales, dtype=dtype)
    want = mx_values(codes, scales).to(dtype)
    assert torch.equal(got[:255], want[:255]) and bool(got[255].isnan().all())


@pytest.mark.parametrize("M,H", [(1, 32), (3, 64), (5, 96), (7, 544), (33, 2048), (2, 8224), (2100, 512), (1, 32768)])
@pytest.mark.parametrize("dtype,pitch", [(torch.bfloat16, 0), (torch.bfloat16, 3), (torch.float32, 0), (torch.float32, 1)], ids=str)
def test_quantize(moe, M, H, dtype, pitch):
    log(f"mxfp4 quantize {M} x {H} {dtype} pitch {pitch}")
    g = gen(M * H)
    x = (torch.randn(M, H + pitch, generator=g, device="cuda") * torch.exp2(torch.randint(-8, 8, (M, 1), generator=g, device="cuda"))).to(dtype)[:, :H]
    codes, scales = moe.moe_mxfp4_quantize(x)
    want, bytes_ = mx_quantised(x)
    assert torch.equal(scales, bytes_) and torch.equal(unsigned_zeros(codes), want)
    assert torch.equal(moe.moe_mxfp4_dequantize(codes, scales).double(), mx_values(codes, scales))


def test_quantize_weights(moe):
    """[E, N, K] gives the pair that the layer's own MXFP4 weights are."""
    w = torch.randn(3, 16, 256, generator=gen(1), device="cuda")
    pair = moe.moe_mxfp4_quantize(w)
    want = mx_quantised(w)
    assert moe.weight_dtype(pair) == moe.MOE_W_MXFP4 and moe.weight_shape(pair) == (3, 16, 256)
    assert torch.equal(pair[1], want[1]) and torch.equal(unsigned_zeros(pair[0]), want[0])
    v = moe.moe_mxfp4_dequantize(*pair, dtype=torch.float32)
    assert v.shape == w.shape and torch.equal(v.double(), mx_values(*pair))


@pytest.mark.parametrize("rows", [r for r in ROWS if not isinstance(r, int)] + [(40, 16, 11, 16, "random", 0.1)], ids=str)
@pytest.mark.parametrize("H", [32, 416, 2080])
def test_quantize_by_expert(moe, rows, H):
    """Codes go where moe_permute takes rows; the other rows stay as they are."""
    log(f"mxfp4 quantize by expert {rows} H={H}")
    r = rows_of(moe, rows, H)
    x = randn(gen(H), r.M, H)
    codes = untouched_buffer(r.rows, H // 2, dtype=torch.uint8)
    scales = untouched_buffer(r.rows, H // MX, dtype=torch.uint8)
    moe.moe_mxfp4_quantize(x, r.perm, r.k, r.rows, codes=codes, scales=scales)
    plain, bytes_ = moe.moe_mxfp4_quantize(x)
    p = r.perm.long()
    assert torch.equal(codes[p[p >= 0]], plain.repeat_interleave(r.k, 0)[p >= 0])
    assert torch.equal(scales[p[p >= 0]], bytes_.repeat_interleave(r.k, 0)[p >= 0])
    assert_untouched(codes, r.kept, "codes")
    assert_untouched(scales, r.kept, "scales")


def test_empty(moe):
    x = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    codes, scales = moe.moe_mxfp4_quantize(x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert moe.moe_mxfp4_dequantize(codes, scales).shape == (0, 64)
    w = mx_weight(gen(1), 1, 64, 64)
    y, _, _ = moe.moe_grouped_linear_mxfp4(x, w)
    assert y.shape == (0, 64)
    assert moe.moe_grouped_linear_mxfp4_backward_x(x, w).shape == (0, 64)


# ---------------------------------------------------------------- products --

def forward_case(moe, rows, act, bias, res, save, rows4, out4, N, K):
    log(f"mxfp4 linear rows={rows} act={act} bias={bias} res={res} save={save} rows4={rows4} out4={out4} N={N} K={K}")
    r = rows_of(moe, rows, N + K)
    g = gen(N * K)
    E, gated = r.E, act == "swiglu"
    w = mx_weight(g, E, N, K)
    up = mx_weight(g, E, N, K) if gated else None
    b = randn(g, E, N) if bias else None
    ub = randn(g, E, N) if bias and gated else None
    if rows4:
        x, xs = mx_rows(g, r.rows, K)
        x64 = mx_values(x, xs)
        xs[~r.kept] = 255  # NaN
    else:
        x, xs = poison(randn(g, r.rows, K), r.kept), None
        x64 = x.double()
    rs = poison(randn(g, r.rows, N), r.kept) if res else None
    out = untouched_buffer(r.rows, N // 2 if out4 else N, dtype=torch.uint8 if out4 else torch.bfloat16)
    out_scale = untouched_buffer(r.rows, N // MX, dtype=torch.uint8) if out4 else None
    pre = untouched_buffer(r.rows, (2 if gated else 1) * N, dtype=torch.bfloat16) if save else None
    y, ys, p = moe.moe_grouped_linear_mxfp4(x, w, r.offsets, r.counts, act=act, up=up, bias=b, up_bias=ub, residual=rs, x_scale=xs,
                                            out=out, out_scale=out_scale, preact=pre)
    torch.cuda.synchronize()
    assert y is out and ys is out_scale and p is pre
    ref, err, pref, perr = reference(r, x64, w, up, b, ub, rs, act)
    k = r.kept
    if out4:
        check_mx_rows(y[k], ys[k], ref[k], err[k], "y")
        assert_untouched(ys, k, "y_scale")
    else:
        assert_within(y[k], ref[k], BF * (ref[k].abs() + err[k]) + err[k] + 1e-37, "y")
    assert_untouched(y, k, "y")
    if save:
        assert_within(pre[k], pref[k], BF * (pref[k].abs() + perr[k]) + perr[k] + 1e-37, "preact")
        assert_untouched(pre, k, "preact")


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("act,bias,res,save", EPILOGUES)
@pytest.mark.parametrize("rows4", [False, True])
@pytest.mark.parametrize("N,K", [(8, 32), (200, 544), (264, 992)])
def test_forward(moe, rows, act, bias, res, save, rows4, N, K):
    forward_case(moe, rows, act, bias, res, save, rows4, False, N, K)


@pytest.mark.parametrize("rows", [1, 300, (70, 6, 3, 16, "skew", 0.1), (260, 4, 2, 16, "random", 0.0)], ids=str)
@pytest.mark.parametrize("act,bias,res,save", EPILOGUES)
@pytest.mark.parametrize("rows4", [False, True])
@pytest.mark.parametrize("N,K", [(32, 64), (224, 416)])
def test_forward_rows_out(moe, rows, act, bias, res, save, rows4, N, K):
    forward_case(moe, rows, act, bias, res, save, rows4, True, N, K)


SKEW = (2100, 16, 4, 16, "skew", 0.0)  # runs of every length, partly filled tiles
# (rows, N, K) that reach every tile, whole and partly filled, with depths that end inside a stage
FORMS = [(33, 544, 288), (64, 160, 2080), ((40, 4, 2, 16, "random", 0.0), 288, 4128), (16, 32, 2208), ((520, 8, 4, 16, "skew", 0.0), 1056, 224),
         (1100, 1056, 224), (2100, 2080, 160), (SKEW, 1056, 160), (4100, 4128, 96), (SKEW, 2080, 256), (SKEW, 1024, 640)]


@pytest.mark.parametrize("rows,N,K", FORMS, ids=str)
@pytest.mark.parametrize("act,bias,res,save", [("gelu", True, True, True), ("swiglu", True, True, True)])
@pytest.mark.parametrize("rows4,out4", [(False, False), (True, False), (False, True), (True, True)])
def test_forward_forms(moe, rows, N, K, act, bias, res, save, rows4, out4):
    forward_case(moe, rows, act, bias, res, save, rows4, out4, N, K)


# 130 experts, three to a lane of a wave, with runs of every length: large tiles in the order of their cost
MANY = (3200, 130, 8, 1, "skew", 0.1)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("rows4,out4", [(False, False), (True, True)])
def test_forward_many_experts(moe, act, rows4, out4):
    forward_case(moe, MANY, act, False, True, False, rows4, out4, 544, 96)


@pytest.mark.parametrize("gated", [False, True])
def test_backward_x_many_experts(moe, gated):
    backward_case(moe, MANY, gated, 72, 1056)


@pytest.mark.parametrize("rows", [5, 200], ids=str)
@pytest.mark.parametrize("rows4", [False, True])
def test_nan_blocks_stay_in_their_rows(moe, rows, rows4):
    """A scale byte of 255 makes its row's (or its column's) results NaN and no other."""
    N, K = 64, 512
    g = gen(7)
    w = mx_weight(g, 1, N, K)
    w[1][0, 9, 3] = 255
    if rows4:
        x, xs = mx_rows(g, rows, K)
        xs[2, 5] = 255
    else:
        x, xs = randn(g, rows, K), None
        x[2, 100] = float("nan")
    y, _, _ = moe.moe_grouped_linear_mxfp4(x, w, x_scale=xs)
    bad = torch.zeros(rows, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 9] = True, True
    assert torch.equal(y.isnan(), bad)
    c, s = moe.moe_grouped_linear_mxfp4(x, w, x_scale=xs, mxfp4_out=True)[:2]
    blocks = bad.reshape(rows, N // MX, MX).any(2)
    assert torch.equal(s == 255, blocks) and bool((c.reshape(rows, -1, MX // 2)[blocks] == 0).all())


def test_scales_far_apart(moe):
    """Blocks whose scales differ by 2^40: the small ones must not shift the large ones."""
    rows, N, K = 64, 32, 1024
    g = gen(11)
    x, xs = mx_rows(g, rows, K)
    w, ws = mx_weight(g, 1, N, K)
    xs += torch.randint(0, 40, xs.shape, generator=g, device="cuda", dtype=torch.uint8)
    ws -= torch.randint(0, 40, ws.shape, generator=g, device="cuda", dtype=torch.uint8)
    xv, wv = mx_values(x, xs), mx_values(w[0], ws[0])
    bound = (K + 8) * SUM * (xv.abs() @ wv.abs().T)
    for a, s in ((x, xs), (moe.moe_mxfp4_dequantize(x, xs), None)):
        y, _, _ = moe.moe_grouped_linear_mxfp4(a, (w, ws), x_scale=s)
        ref = xv @ wv.T
        assert_within(y, ref, BF * (ref.abs() + bound) + bound)


def test_unaligned_scale_bytes(moe):
    """Scale bytes may begin anywhere."""
    rows, N, K = 150, 96, 416
    g = gen(13)
    x, xs = mx_rows(g, rows, K)
    w, ws = mx_weight(g, 1, N, K)

    def shifted(t):
        flat = torch.zeros(t.numel() + 3, dtype=torch.uint8, device="cuda")
        v = flat[3:].view(t.shape)
        v.copy_(t)
        return v

    a = moe.moe_grouped_linear_mxfp4(x, (w, ws), x_scale=xs, mxfp4_out=True)
    b = moe.moe_grouped_linear_mxfp4(x, (w, shifted(ws)), x_scale=shifted(xs), mxfp4_out=True, out_scale=shifted(a[1] * 0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dz = randn(g, rows, N)
    assert torch.equal(moe.moe_grouped_linear_mxfp4_backward_x(dz, (w, ws)), moe.moe_grouped_linear_mxfp4_backward_x(dz, (w, shifted(ws))))


# ----------------------------------------------------------- rows' gradient --

def backward_case(moe, rows, gated, N, K):
    log(f"mxfp4 backward x rows={rows} gated={gated} N={N} K={K}")
    r = rows_of(moe, rows, N + K)
    g = gen(N * K + 3)
    wide = 2 if gated else 1
    dz = poison(randn(g, r.rows, wide * N), r.kept)
    w = mx_weight(g, r.E, N, K)
    up = mx_weight(g, r.E, N, K) if gated else None
    dx = untouched_buffer(r.rows, K, dtype=torch.bfloat16)
    assert moe.moe_grouped_linear_mxfp4_backward_x(dz, w, r.offsets, r.counts, up=up, dx=dx) is dx
    torch.cuda.synchronize()
    for e, at, n in r.runs:
        if n == 0:
            continue
        m = mx_values(w[0][e], w[1][e])
        if gated:
            m = torch.cat([m, mx_values(up[0][e], up[1][e])])
        d = dz[at:at + n].double()
        ref, err = d @ m, (wide * N + 8) * SUM * (d.abs() @ m.abs())
        assert_within(dx[at:at + n], ref, BF * (ref.abs() + err) + err + 1e-37, "dx")
    assert_untouched(dx, r.kept, "dx")


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(8, 32), (200, 544), (264, 992)])
def test_backward_x(moe, rows, gated, N, K):
    backward_case(moe, rows, gated, N, K)


@pytest.mark.parametrize("rows,N,K", [(1100, 200, 1056), (SKEW, 136, 1056), (4100, 72, 4128), (SKEW, 200, 2080), (64, 1032, 96), (16, 2056, 160),
                                      ((40, 4, 2, 16, "random", 0.0), 1032, 288)], ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_backward_x_forms(moe, rows, N, K, gated):
    backward_case(moe, rows, gated, N, K)


def test_backward_x_against_differences(moe):
    """The loss <c, W x> moves by <dx, v> along v: exact up to the rounding of dx and of
    the products, whose bounds are summed over v."""
    rows, N, K = 40, 72, 160
    g = gen(21)
    x, v, c = (randn(g, rows, n) for n in (K, K, N))
    w = mx_weight(g, 1, N, K)
    dx = moe.moe_grouped_linear_mxfp4_backward_x(c, w).double()
    m = mx_values(w[0][0], w[1][0])
    y = [moe.moe_grouped_linear_mxfp4(t, w)[0].double() for t in ((x.double() + v.double()).bfloat16(), x)]
    step = (x.double() + v.double()).bfloat16().double() - x.double()
    moved = ((y[0] - y[1]) * c.double()).sum()
    terms = [(t.double().abs() @ m.abs().T) for t in ((x.double() + v.double()).bfloat16(), x)]
    bound = sum(((BF * t + (K + 8) * SUM * t) * c.double().abs()).sum() for t in terms)
    bound += ((BF + (N + 8) * SUM) * (c.double().abs() @ m.abs()) * step.abs()).sum()
    assert float((moved - (dx * step).sum()).abs()) <= float(bound)
