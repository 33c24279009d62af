"""The experts' products over sorted rows and their gradients against the formulas
in float64 (bounds: see ops_testlib)."""

import math

import pytest
import torch

from moe_testlib import log
from ops_testlib import (BLOCK, SUM, Dense, Routed, assert_untouched, assert_within, check_fp8_rows, dequantised, gen, half,
                         poison, quantised, randn, untouched_buffer)

pytestmark = pytest.mark.gpu

BF = half(torch.bfloat16)
# largest slope of silu and gelu, and of their derivatives
SLOPE, CURVE = 1.13, 1.0
# float32 evaluation of the activations: a few roundings of values of their size
ACT = 16 * SUM


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def rows_of(moe, kind, seed):
    if isinstance(kind, int):
        return Dense(kind)
    M, E, k, BS, mode, drop = kind
    return Routed(moe, M, E, k, BS, seed, mode, drop)


def fp8_weight(g, E, N, K):
    v = torch.randn(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK, generator=g, device="cuda") * K ** -0.5
    scale = v.abs().amax((2, 4)) / 448
    return (v / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).reshape(E, N, K).view(torch.uint8), scale.contiguous()


def weight64(w, e):
    codes, scale = w
    if scale is None:
        return codes[e].double()
    return codes[e].view(torch.float8_e4m3fn).double() * scale[e].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


def act64(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def reference(r, x, w, up, bias, up_bias, residual, act):
    """y, its error bound before the last rounding, and the pre-activations with theirs."""
    N, K = w[0].shape[1:]
    wide = 1 if up is None else 2
    y = torch.zeros(r.rows, N, dtype=torch.float64, device="cuda")
    yerr, pre = torch.zeros_like(y), torch.zeros(r.rows, wide * N, dtype=torch.float64, device="cuda")
    perr = torch.zeros_like(pre)
    for e, at, n in r.runs:
        if n == 0:
            continue
        s = slice(at, at + n)

        def product(weights, b):
            m = weight64(weights, e)
            z, mag = x[s] @ m.T, x[s].abs() @ m.abs().T
            if b is not None:
                z, mag = z + b[e].double(), mag + b[e].double().abs()
            return z, (K + 8) * SUM * mag

        z, ze = product(w, bias)
        pre[s, :N], perr[s, :N] = z, ze
        if up is not None:
            u, ue = product(up, up_bias)
            pre[s, N:], perr[s, N:] = u, ue
            a = act64("silu", z)
            v, ve = a * u, SLOPE * ze * (u.abs() + ue) + a.abs() * ue + ACT * (a * u).abs()
        else:
            v = act64(act, z)
            ve = (SLOPE * ze + ACT * v.abs()) if act != "none" else ze
        if residual is not None:
            v = v + residual[s].double()
            ve = ve + SUM * v.abs()
        y[s], yerr[s] = v, ve
    return y, yerr, pre, perr


ROWS = [
    1, 17, 300,                              # dense
    (1, 8, 2, 16, "random", 0.0),            # one token
    (5, 300, 4, 1, "random", 0.3),           # more experts than lanes
    (70, 6, 3, 16, "skew", 0.1),             # experts without a row
    (150, 3, 2, 64, "one", 0.0),             # one expert holds everything
    (260, 4, 2, 16, "random", 0.0),          # runs that end inside a tile
    (9, 5, 2, 16, "random", 1.0),            # no row at all
]
# act, bias, residual, preact
EPILOGUES = [("none", False, False, False), ("none", True, True, False), ("silu", True, False, True),
             ("gelu", True, True, True), ("swiglu", False, False, True), ("swiglu", True, True, False)]


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("act,bias,res,save", EPILOGUES)
@pytest.mark.parametrize("N,K", [(8, 8), (200, 520), (264, 1000)])
def test_forward(moe, rows, act, bias, res, save, N, K):
    log(f"linear rows={rows} act={act} bias={bias} res={res} save={save} N={N} K={K}")
    r = rows_of(moe, rows, N + K)
    g = gen(N * K)
    E, gated = r.E, act == "swiglu"
    x = poison(randn(g, r.rows, K), r.kept)
    w = (randn(g, E, N, K, scale=K ** -0.5), None)
    up = (randn(g, E, N, K, scale=K ** -0.5), None) if gated else None
    b = randn(g, E, N) if bias else None
    ub = randn(g, E, N) if bias and gated else None
    rs = poison(randn(g, r.rows, N), r.kept) if res else None
    out = untouched_buffer(r.rows, N, dtype=torch.bfloat16)
    pre = untouched_buffer(r.rows, (2 if gated else 1) * N, dtype=torch.bfloat16) if save else None
    y, none, p = moe.moe_grouped_linear(x, w, r.offsets, r.counts, act=act, up=up, bias=b, up_bias=ub, residual=rs, out=out,
                                        preact=pre)
    torch.cuda.synchronize()
    assert none is None and y is out and p is pre
    ref, err, pref, perr = reference(r, x.double(), w, up, b, ub, rs, act)
    k = r.kept
    assert_within(y[k], ref[k], BF * (ref[k].abs() + err[k]) + err[k] + 1e-37, "y")
    assert_untouched(y, k, "y")
    if save:
        assert_within(pre[k], pref[k], BF * (pref[k].abs() + perr[k]) + perr[k] + 1e-37, "preact")
        assert_untouched(pre, k, "preact")


@pytest.mark.parametrize("rows", [1, 40, (1, 8, 2, 16, "random", 0.0), (70, 6, 3, 16, "skew", 0.1),
                                  (260, 4, 2, 16, "random", 0.0), (9, 5, 2, 16, "random", 1.0)], ids=str)
@pytest.mark.parametrize("act,bias,res,fp8_out", [("none", False, False, False), ("none", True, True, True),
                                                  ("gelu", False, False, True), ("swiglu", False, False, True),
                                                  ("swiglu", True, True, False)])
@pytest.mark.parametrize("N,K", [(128, 128), (384, 640)])
def test_forward_8bit(moe, rows, act, bias, res, fp8_out, N, K):
    log(f"linear 8-bit rows={rows} act={act} bias={bias} res={res} out8={fp8_out} N={N} K={K}")
    r = rows_of(moe, rows, N + K)
    g = gen(N * K + 1)
    E, gated = r.E, act == "swiglu"
    xs, x_scale = quantised(randn(g, r.rows, K))
    x64 = dequantised(xs, x_scale)
    poison(xs, r.kept)
    poison(x_scale, r.kept)
    w = fp8_weight(g, E, N, K)
    up = fp8_weight(g, E, N, K) if gated else None
    b = randn(g, E, N) if bias else None
    ub = randn(g, E, N) if bias and gated else None
    rs = poison(randn(g, r.rows, N), r.kept) if res else None
    out = untouched_buffer(r.rows, N, dtype=torch.float8_e4m3fn if fp8_out else torch.bfloat16)
    out_scale = untouched_buffer(r.rows, N // BLOCK, dtype=torch.float32) if fp8_out else None
    moe.moe_grouped_linear(xs, w, r.offsets, r.counts, act=act, up=up, bias=b, up_bias=ub, residual=rs, x_scale=x_scale, out=out,
                           out_scale=out_scale)
    torch.cuda.synchronize()
    ref, err, _, _ = reference(r, x64, w, up, b, ub, rs, act)
    k = r.kept
    if fp8_out:
        check_fp8_rows(out.view(torch.uint8)[k], out_scale[k], ref[k], err[k], "y")
        assert_untouched(out_scale, k, "y_scale")
    else:
        assert_within(out[k], ref[k], BF * (ref[k].abs() + err[k]) + err[k] + 1e-37, "y")
    assert_untouched(out, k, "y")


# (rows, N, K) that reach the 256-wide tiles and the depth-split kernel of a few rows, whole and partly filled
WIDE = [(1100, 2048, 264), ((520, 8, 4, 16, "skew", 0.0), 1040, 200), ((700, 6, 4, 1, "random", 0.1), 1032, 136),
        (33, 520, 264), (64, 136, 2056), ((40, 4, 2, 16, "random", 0.0), 264, 4104), (16, 24, 2184)]


@pytest.mark.parametrize("rows,N,K", WIDE, ids=str)
@pytest.mark.parametrize("act,bias,res,save", [("none", True, True, False), ("swiglu", True, False, True)])
def test_forward_tiles(moe, rows, N, K, act, bias, res, save):
    test_forward(moe, rows, act, bias, res, save, N, K)


SKEW = (2100, 16, 4, 16, "skew", 0.0)  # runs of every length, partly filled tiles
# (rows, N, K) by the tiles they take without SwiGLU: 64 x 64, 128 x 128, 256 x 256
FORMS = [(1100, 1040, 200), (2100, 2056, 136), (SKEW, 1032, 136), (4100, 4104, 72), (SKEW, 2056, 200)]


@pytest.mark.parametrize("rows,N,K", FORMS, ids=str)
@pytest.mark.parametrize("act,bias,res,save", [("gelu", True, True, True), ("swiglu", True, True, True)])
def test_forward_forms(moe, rows, N, K, act, bias, res, save):
    test_forward(moe, rows, act, bias, res, save, N, K)


@pytest.mark.parametrize("rows,N,K", [(1100, 1024, 256), (2100, 2048, 128), (SKEW, 1024, 384)], ids=str)
@pytest.mark.parametrize("act,bias,res", [("gelu", True, True), ("swiglu", True, True)])
def test_forward_8bit_forms(moe, rows, N, K, act, bias, res):
    test_forward_8bit(moe, rows, act, bias, res, False, N, K)


# the rows' gradient by 64 x 128, 128 x 128 and 256 x 256 tiles
@pytest.mark.parametrize("rows,N,K", [(1100, 200, 1032), (SKEW, 136, 1032), (4100, 72, 4104), (SKEW, 200, 2056)], ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_backward_forms(moe, rows, N, K, gated):
    test_backward(moe, rows, gated, N, K)


@pytest.mark.parametrize("rows", [1, 40, 300, (70, 6, 3, 16, "skew", 0.1), (600, 4, 2, 16, "random", 0.0)], ids=str)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("N,K", [(128, 136), (640, 520)])
def test_bf16_operands_to_8bit_rows(moe, rows, act, N, K):
    r = rows_of(moe, rows, N)
    g = gen(N + K)
    gated = act == "swiglu"
    x = poison(randn(g, r.rows, K), r.kept)
    w = (randn(g, r.E, N, K, scale=K ** -0.5), None)
    up = (randn(g, r.E, N, K, scale=K ** -0.5), None) if gated else None
    out = untouched_buffer(r.rows, N, dtype=torch.float8_e4m3fn)
    out_scale = untouched_buffer(r.rows, N // BLOCK, dtype=torch.float32)
    moe.moe_grouped_linear(x, w, r.offsets, r.counts, act=act, up=up, out=out, out_scale=out_scale)
    torch.cuda.synchronize()
    ref, err, _, _ = reference(r, x.double(), w, up, None, None, None, act)
    k = r.kept
    check_fp8_rows(out.view(torch.uint8)[k], out_scale[k], ref[k], err[k], "y")
    assert_untouched(out, k, "y")
    assert_untouched(out_scale, k, "y_scale")


@pytest.mark.parametrize("rows", [1, 33, 300, (700, 6, 4, 1, "skew", 0.1)], ids=str)
@pytest.mark.parametrize("fp8_out", [False, True])
def test_8bit_wide_depth(moe, rows, fp8_out):
    """Scales of a small and a large block stay exact to float32 sums: each scale
    holds to the bound of the products."""
    test_forward_8bit(moe, rows, "swiglu", False, False, fp8_out, 256, 2048)


@pytest.mark.parametrize("rows,N,K,gated", [((520, 32, 4, 16, "skew", 0.0), 1040, 520, False),
                                            ((300, 16, 4, 16, "random", 0.0), 600, 1032, True)], ids=str)
def test_backward_tiles(moe, rows, N, K, gated):
    test_backward(moe, rows, gated, N, K)


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(8, 8), (200, 520), (520, 264)])
def test_backward(moe, rows, gated, N, K):
    log(f"linear backward rows={rows} gated={gated} N={N} K={K}")
    r = rows_of(moe, rows, N + K)
    g = gen(N + 3 * K)
    E, parts = r.E, 2 if gated else 1
    x = poison(randn(g, r.rows, K), r.kept)
    dz = poison(randn(g, r.rows, parts * N), r.kept)
    ws = [randn(g, E, N, K, scale=N ** -0.5) for _ in range(parts)]
    dx = untouched_buffer(r.rows, K, dtype=torch.bfloat16)
    moe.moe_grouped_linear_backward_x(dz, ws[0], r.offsets, r.counts, up=ws[1] if gated else None, dx=dx)
    for kind in (torch.bfloat16, torch.float32):
        grads = moe.moe_grouped_linear_backward_w(dz, x, r.offsets, r.counts, gated=gated, bias=True, dtype=kind)
        torch.cuda.synchronize()
        for h in range(parts):
            dw, db = grads[h], grads[2 + h]
            for e, at, n in r.runs:
                d, xx = dz[at:at + n, h * N:(h + 1) * N].double(), x[at:at + n].double()
                ref, mag = d.T @ xx, d.abs().T @ xx.abs()
                assert_within(dw[e], ref, half(kind) * ref.abs() + (n + 8) * SUM * mag, f"dw[{h}][{e}]")
                assert_within(db[e], d.sum(0), (n + 8) * SUM * d.abs().sum(0), f"db[{h}][{e}]")
    refx = torch.zeros(r.rows, K, dtype=torch.float64, device="cuda")
    magx = torch.zeros_like(refx)
    for e, at, n in r.runs:
        for h in range(parts):
            d = dz[at:at + n, h * N:(h + 1) * N].double()
            refx[at:at + n] += d @ ws[h][e].double()
            magx[at:at + n] += d.abs() @ ws[h][e].double().abs()
    k = r.kept
    assert_within(dx[k], refx[k], BF * refx[k].abs() + (parts * N + 8) * SUM * magx[k] + 1e-37, "dx")
    assert_untouched(dx, k, "dx")


@pytest.mark.parametrize("rows", [1, 300, (70, 6, 3, 16, "skew", 0.1), (9, 5, 2, 16, "random", 1.0)], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("N", [8, 200])
def test_act_backward(moe, rows, act, N):
    r = rows_of(moe, rows, N)
    g = gen(N + len(act))
    wide = 2 if act == "swiglu" else 1
    pre = randn(g, r.rows, wide * N, scale=2.0)
    pre[0, :8] = torch.tensor([0.0, -0.0, 80.0, -80.0, 1e-30, 3e38, -3e38, 5.0], device="cuda")
    pre, dy = poison(pre, r.kept), poison(randn(g, r.rows, N), r.kept)
    dz = untouched_buffer(r.rows, wide * N, dtype=torch.bfloat16)
    moe.moe_grouped_act_backward(dy, pre, act, r.offsets, r.counts, dz=dz)
    torch.cuda.synchronize()
    k = r.kept
    z = pre[k][:, :N].double().requires_grad_()
    a = act64("silu" if act == "swiglu" else act, z)
    slope = torch.autograd.grad(a.sum(), z)[0]
    z, a, d = z.detach(), a.detach(), dy[k].double()
    if act == "gelu":  # the formula's cube overflows past 1e102 nowhere, but its slope there is 0 or 1
        slope = torch.where(z.abs() > 30, (z > 0).double(), slope)
    # the slope is made of terms of the size 1 + |z| s(1 - s), which is below 2
    if act == "swiglu":
        u = pre[k][:, N:].double()
        ref, mag = torch.cat([d * u * slope, d * a], 1), torch.cat([2 * (d * u).abs(), (d * a).abs()], 1)
    else:
        ref, mag = d * slope, 2 * d.abs()
    # dy * z reaches past bf16's largest value, (2 - 2^-7) 2^127; from half a step above
    # it, (2 - 2^-8) 2^127, round to nearest gives an infinity of that sign
    past = ref.abs() >= (2 - 2.0 ** -8) * 2.0 ** 127
    assert torch.equal(dz[k][past].double(), torch.copysign(torch.full_like(ref[past], math.inf), ref[past]))
    assert_within(torch.where(past, 0.0, dz[k].double()), torch.where(past, 0.0, ref), BF * ref.abs() + ACT * mag + 1e-37, "dz")
    assert_untouched(dz, k, "dz")
    moe.moe_grouped_act_backward(dy, pre, act, r.offsets, r.counts, dz=pre)  # over its own input
    assert torch.equal(pre[k], dz[k])


def test_runs_past_the_matrix_are_cut(moe):
    """Offsets and counts that reach past the rows, or are negative, name no row there."""
    N, K, rows = 64, 64, 40
    g = gen(4)
    x, w, dz = randn(g, rows, K), randn(g, 4, N, K, scale=0.1), randn(g, rows, N)
    offsets = torch.tensor([0, 30, 50, -5, 60], dtype=torch.int32, device="cuda")
    counts = torch.tensor([10, 20, 8, 6], dtype=torch.int32, device="cuda")
    out = untouched_buffer(rows, N, dtype=torch.bfloat16)
    moe.moe_grouped_linear(x, w, offsets, counts, out=out)
    dw, _, db, _ = moe.moe_grouped_linear_backward_w(dz, x, offsets, counts, bias=True)
    torch.cuda.synchronize()
    kept = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, at, n in ((0, 0, 10), (1, 30, 10)):
        kept[at:at + n] = True
        ref = x[at:at + n].double() @ w[e].double().T
        assert_within(out[at:at + n], ref, BF * ref.abs() + K * SUM * (x[at:at + n].double().abs() @ w[e].double().abs().T))
        ref = dz[at:at + n].double().sum(0)
        assert_within(db[e], ref, 20 * SUM * dz[at:at + n].double().abs().sum(0))
    assert_untouched(out, kept)
    assert not bool(dw[2:].any()) and not bool(db[2:].any())


@pytest.mark.parametrize("rows,N", [(700, 8), (5000, 136), (20000, 64)])
def test_runs_that_overlap_stay_in_bounds(moe, rows, N):
    """Every expert claims every row: far more tiles than the rows can make.  The
    tiles past that are left out and nothing behind the matrix is written; all
    experts hold the same weights, so whichever of them takes a row gives its value."""
    E, K = 1024, 16
    g = gen(6)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    counts = torch.full((E,), rows + 5, dtype=torch.int32, device="cuda")
    x, dz = randn(g, rows, K), randn(g, rows, N)
    w = randn(g, 1, N, K).expand(E, N, K).contiguous()
    pre = randn(g, rows, N)
    guard = 300
    whole = [untouched_buffer(rows + guard, c, dtype=torch.bfloat16) for c in (N, K, N)]
    y, dx, da = (t[:rows] for t in whole)
    moe.moe_grouped_linear(x, w, offsets, counts, out=y)
    moe.moe_grouped_linear_backward_x(dz, w, offsets, counts, dx=dx)
    moe.moe_grouped_act_backward(dz, pre, "silu", offsets, counts, dz=da)
    torch.cuda.synchronize()
    kept = torch.arange(rows + guard, device="cuda") < rows
    for t in whole:
        assert_untouched(t, kept)
    wd, zd, xd = w[0].double(), dz.double(), x.double()
    for got, ref, mag, depth in ((y, xd @ wd.T, xd.abs() @ wd.abs().T, K), (dx, zd @ wd, zd.abs() @ wd.abs(), N)):
        assert_within(got, ref, BF * ref.abs() + depth * SUM * mag)
    p = pre.double()
    sg = torch.sigmoid(p)
    ref = zd * sg * (1 + p * (1 - sg))
    assert_within(da, ref, BF * ref.abs() + ACT * zd.abs() * (1 + p.abs()))


def test_in_place_residual_and_repeat(moe):
    """y over the residual's buffer, and the same bits on every call."""
    g = gen(9)
    x, w, rs = randn(g, 50, 264), randn(g, 1, 136, 264, scale=0.1), randn(g, 50, 136)
    a, _, _ = moe.moe_grouped_linear(x, w, residual=rs)
    for _ in range(3):
        assert torch.equal(moe.moe_grouped_linear(x, w, residual=rs)[0], a)
    b, _, _ = moe.moe_grouped_linear(x, w, residual=rs, out=rs)
    assert torch.equal(a, b)


def test_large_dense_gradient_splits_rows(moe):
    """A small weight over many rows: the row splits join to the same sums."""
    rows, N, K = 5000, 72, 40
    g = gen(1)
    dz, x = randn(g, rows, N), randn(g, rows, K)
    assert moe.lib().moe_grouped_linear_backward_w_workspace_bytes(rows, 1, N, K, 0, 1) > 0
    dw, _, db, _ = moe.moe_grouped_linear_backward_w(dz, x, bias=True, dtype=torch.float32)
    d, xx = dz.double(), x.double()
    assert_within(dw[0], d.T @ xx, (rows + 8) * SUM * (d.abs().T @ xx.abs()))
    assert_within(db[0], d.sum(0), (rows + 8) * SUM * d.abs().sum(0))


def test_graph_replay(moe):
    M, E, k, N, K = 90, 6, 2, 136, 264
    r = Routed(moe, M, E, k, 16, 1)
    g = gen(2)
    x, dz = randn(g, r.rows, K), randn(g, r.rows, 2 * N)
    w, up = randn(g, E, N, K, scale=0.1), randn(g, E, N, K, scale=0.1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        y, _, pre = moe.moe_grouped_linear(x, w, r.offsets, r.counts, act="swiglu", up=up, save_preact=True,
                                           out=torch.zeros(r.rows, N, dtype=torch.bfloat16, device="cuda"),
                                           preact=torch.zeros(r.rows, 2 * N, dtype=torch.bfloat16, device="cuda"))
        d = moe.moe_grouped_act_backward(y, pre, "swiglu", r.offsets, r.counts, dz=torch.zeros_like(pre))
        dx = moe.moe_grouped_linear_backward_x(dz, w, r.offsets, r.counts, up=up, dx=torch.zeros_like(x))
        return (y, pre, d, dx) + moe.moe_grouped_linear_backward_w(dz, x, r.offsets, r.counts, gated=True, bias=True)

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    for seed in (1, 2, 3):
        n = Routed(moe, M, E, k, 16, 20 + seed, drop=0.1)
        r.offsets.copy_(n.offsets)
        r.counts.copy_(n.counts)
        x.copy_(randn(gen(seed), r.rows, K))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_biases_are_independent(moe):
    """Either bias of a gated product may be left out."""
    g = gen(3)
    r = Routed(moe, 60, 4, 2, 16, 1)
    N, K = 72, 136
    x, w, up = poison(randn(g, r.rows, K), r.kept), (randn(g, 4, N, K, scale=0.1), None), (randn(g, 4, N, K, scale=0.1), None)
    b = randn(g, 4, N)
    for bias, up_bias in ((b, None), (None, b)):
        y, _, _ = moe.moe_grouped_linear(x, w, r.offsets, r.counts, act="swiglu", up=up, bias=bias, up_bias=up_bias)
        ref, err, _, _ = reference(r, x.double(), w, up, bias, up_bias, None, "swiglu")
        k = r.kept
        assert_within(y[k], ref[k], BF * (ref[k].abs() + err[k]) + err[k] + 1e-37, "y")


def test_rows_of_a_tile_do_not_mix(moe):
    """A NaN or an infinity in one row stays in that row's results, whole and partly
    filled tiles alike; far activations keep their limits."""
    g = gen(8)
    for rows in (20, 300, 1000):
        x, w = randn(g, rows, 264), randn(g, 1, 520, 264, scale=0.1)
        a, _, _ = moe.moe_grouped_linear(x, w, act="silu")
        x[7] = float("nan")
        x[rows - 1, 3] = float("inf")
        b, _, _ = moe.moe_grouped_linear(x, w, act="silu")
        torch.cuda.synchronize()
        assert bool(b[7].isnan().all())
        rest = [i for i in range(rows) if i not in (7, rows - 1)]
        assert torch.equal(a[rest], b[rest])
    # identity weights: z itself through the activations
    z = torch.tensor([0.0, -0.0, 90.0, -90.0, 3e38, -3e38, float("inf"), float("nan")], device="cuda").to(torch.bfloat16)
    eye = torch.eye(8, device="cuda").to(torch.bfloat16)[None]
    x = torch.diag(z.nan_to_num(1.0, 1.0)).to(torch.bfloat16)
    for act in ("silu", "gelu"):
        y, _, _ = moe.moe_grouped_linear(x, eye, act=act)
        d = torch.diagonal(y).float()
        assert d[0] == 0 and d[1] == 0 and d[2] == 90 and abs(float(d[3])) < 1e-35 and d[4] == z[4].float() and d[5] == 0, act
