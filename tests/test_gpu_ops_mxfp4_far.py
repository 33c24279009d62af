"""The 4-bit operators past 32 bits: matrices whose byte offsets pass 2^32, 2^31 - 1 rows,
and more workgroups than one grid dimension holds."""

import pytest
import torch

from moe_testlib import log
from mx_testlib import mx_quantised, mx_values, mx_weight
from ops_testlib import SUM, gen, half, randn

pytestmark = pytest.mark.gpu

BF = half(torch.bfloat16)
TAIL = 300


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of GPU memory")


def test_far_rows(moe):
    rows, K, N = 600_000, 8192, 32  # 9.8 GB of bf16 rows, 2.5 GB of codes
    log(f"4-bit products of {rows} x {K}")
    need(40)
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    w = mx_weight(gen(2), 2, N, K)
    split = rows - TAIL
    offsets = torch.tensor([0, split, rows], dtype=torch.int32, device="cuda")
    counts = torch.tensor([split, TAIL], dtype=torch.int32, device="cuda")
    codes, scales = moe.moe_mxfp4_quantize(x)
    want = mx_quantised(x[split:])
    v = mx_values(*want)
    assert torch.equal(mx_values(codes[split:], scales[split:]), v)
    assert torch.equal(moe.moe_mxfp4_dequantize(codes, scales)[split:].double(), v)
    m = mx_values(w[0][1], w[1][1])
    for a, s, a64 in ((x, None, x[split:].double()), (codes, scales, v)):
        y, _, _ = moe.moe_grouped_linear_mxfp4(a, w, offsets, counts, x_scale=s)
        ref, mag = a64 @ m.T, a64.abs() @ m.abs().T
        assert bool(((y[split:].double() - ref).abs() <= BF * ref.abs() + 2 * (K + 8) * SUM * mag).all())
    dx = moe.moe_grouped_linear_mxfp4_backward_x(y, w, offsets, counts)
    d = y[split:].double()
    assert bool(((dx[split:].double() - d @ m).abs() <= BF * (d @ m).abs() + 2 * (N + 8) * SUM * (d.abs() @ m.abs()) + 1e-37).all())


@pytest.mark.parametrize("grouped", [False, True])
def test_most_rows(moe, grouped):
    rows, K, N = 2 ** 31 - 1, 32, 8  # 34 GB of codes, 34 GB of results, 137 GB of gradients
    log(f"4-bit products of {rows} rows, grouped={grouped}")
    need(230)
    x, s = mx_quantised(torch.ones(1, K, device="cuda"))
    codes, scales = x.expand(rows, -1).contiguous(), s.expand(rows, -1).contiguous()
    ends = [slice(0, TAIL), slice(rows - TAIL, rows)]
    for i, part in enumerate(ends):
        codes[part], scales[part] = mx_quantised(randn(gen(i), TAIL, K))
    w = mx_weight(gen(5), 1, N, K)
    m = mx_values(w[0][0], w[1][0])
    runs = ()
    if grouped:
        runs = (torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.tensor([rows], dtype=torch.int32, device="cuda"))
    y = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_mxfp4(codes, w, *runs, x_scale=scales, out=y)
    torch.cuda.synchronize()
    for part in ends:
        a = mx_values(codes[part], scales[part])
        assert bool(((y[part].double() - a @ m.T).abs() <= BF * (a @ m.T).abs() + 64 * SUM * (a.abs() @ m.abs().T)).all())
    step = 1 << 27
    for at in range(TAIL, rows - TAIL, step):
        assert bool((y[at:min(at + step, rows - TAIL)] == y[TAIL]).all()), at
    del codes, scales
    log("rows' gradient")
    dx = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_mxfp4_backward_x(y, w, *runs, dx=dx)
    torch.cuda.synchronize()
    for part in ends:
        d = y[part].double()
        assert bool(((dx[part].double() - d @ m).abs() <= BF * (d @ m).abs() + 32 * SUM * (d.abs() @ m.abs()) + 1e-37).all())
    for at in range(TAIL, rows - TAIL, step):
        assert bool((dx[at:min(at + step, rows - TAIL)] == dx[TAIL]).all()), at


@pytest.mark.parametrize("H", [32, 544])  # 4 and 64 threads a row
def test_many_rows(moe, H):
    M = (64 if H == 32 else 4) * 2 ** 21 + 37
    log(f"mxfp4 quantize {M} x {H}")
    need(60)
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(3))
    perm = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    codes, scales = moe.moe_mxfp4_quantize(x, perm, 1, M)
    back = moe.moe_mxfp4_dequantize(codes, scales)
    for part in (slice(0, TAIL), slice(M - TAIL, M)):
        assert torch.equal(back.flip(0)[part].double() if M < 10_000_000 else back[M - part.stop:M - part.start].flip(0).double(), mx_values(*mx_quantised(x[part])))
    plain, bytes_ = moe.moe_mxfp4_quantize(x)
    assert torch.equal(plain[-TAIL:].flip(0), codes[:TAIL]) and torch.equal(bytes_[:TAIL].flip(0), scales[-TAIL:])


def test_many_experts(moe):
    """1024 experts, most without a row, one of them with nearly all."""
    E, N, K = 1024, 96, 160
    g = gen(9)
    counts = torch.randint(0, 3, (E,), generator=g, device="cuda", dtype=torch.int32)
    counts[777] = 900
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    rows = int(offsets[-1])
    x = randn(g, rows, K)
    w = mx_weight(g, E, N, K)
    q, s = moe.moe_mxfp4_quantize(x)
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
    wv = mx_values(*w)
    for a, xs, v in ((x, None, x.double()), (q, s, mx_values(q, s))):
        y, _, _ = moe.moe_grouped_linear_mxfp4(a, w, offsets, counts, x_scale=xs)
        ref = torch.stack([wv[owner[i]] @ v[i] for i in range(rows)])
        mag = torch.stack([wv[owner[i]].abs() @ v[i].abs() for i in range(rows)])
        assert bool(((y.double() - ref).abs() <= BF * ref.abs() + 2 * (K + 8) * SUM * mag).all())


def test_far_gradients(moe):
    """A tensor past 2^32 bytes beside a small one."""
    n = 2_300_000_011
    log(f"clip {n} gradients")
    need(20)
    g = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    small = torch.full((5,), 3.0, device="cuda")
    g[-1] = 100.0
    norm = moe.moe_clip_grad_norm([g, small], 10.0)
    want = ((n - 1) * 2.0 ** -20 + 1e4 + 45.0) ** 0.5
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    c = 10.0 / want
    for v, ref in ((g[0], 2.0 ** -10), (g[n // 2], 2.0 ** -10), (g[-2], 2.0 ** -10), (g[-1], 100.0)):
        assert abs(float(v) - ref * c) <= ref * c * 2.0 ** -8
    assert bool((g[:-1] == g[0]).all()) and bool(((small - 3.0 * c).abs() <= 2.0 ** -21).all())
