"""An expert block whose experts are held in 4 bits: a training step on float32 master
weights (rounded, products, gradients straight through the rounding, clipped) against
float64 autograd, the serving chain in 4 bits stage by stage, graph replays, two streams,
and the layer kernels on the same weights."""

import math
import os
import re

import pytest
import torch

from moe_testlib import log
from mx_testlib import check_mx_rows, mx_quantised, mx_values, mx_weight, reference
from ops_testlib import Routed, assert_within, gen, half, randn
from test_gpu_ops_chain import EPS, close

pytestmark = pytest.mark.gpu

STEP = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


class Block:
    """float32 master weights of the experts, and the rows of one step."""

    def __init__(self, M, H, I, E, seed):
        g = gen(seed)
        self.x, self.res, self.dout = randn(g, M, H), randn(g, M, H), randn(g, M, H)
        self.nw = randn(g, H, scale=0.1) + 1.0
        f32 = torch.float32
        self.gate, self.up = randn(g, E, I, H, scale=H ** -0.5, dtype=f32), randn(g, E, I, H, scale=H ** -0.5, dtype=f32)
        self.down = randn(g, E, H, I, scale=I ** -0.5, dtype=f32)


def train(moe, b, r, max_norm):
    """One step up to the clipped gradients, which are scaled in place."""
    gate, up, down = (moe.moe_mxfp4_quantize(w) for w in (b.gate, b.up, b.down))
    n, _, z, rstd = moe.moe_add_rms_norm(b.x, b.nw, EPS, residual=b.res, save_rstd=True)
    xs, _ = moe.moe_permute(n, r.perm, r.k, r.rows)
    h, _, pre = moe.moe_grouped_linear_mxfp4(xs, gate, r.offsets, r.counts, act="swiglu", up=up, save_preact=True)
    y, _, _ = moe.moe_grouped_linear_mxfp4(h, down, r.offsets, r.counts)
    out = moe.moe_unpermute(y, r.perm, r.k, topk_weights=r.weights)
    dy, dwts = moe.moe_unpermute_backward(b.dout, y, r.perm, r.weights)
    dh = moe.moe_grouped_linear_mxfp4_backward_x(dy, down, r.offsets, r.counts)
    ddown, _, _, _ = moe.moe_grouped_linear_backward_w(dy, h, r.offsets, r.counts, dtype=torch.float32)
    dz = moe.moe_grouped_act_backward(dh, pre, "swiglu", r.offsets, r.counts)
    dgate, dup, _, _ = moe.moe_grouped_linear_backward_w(dz, xs, r.offsets, r.counts, gated=True)
    dn = moe.moe_unpermute(moe.moe_grouped_linear_mxfp4_backward_x(dz, gate, r.offsets, r.counts, up=up), r.perm, r.k)
    dx, dnw = moe.moe_add_rms_norm_backward(dn, z, b.nw, rstd, dz=b.dout)
    grads = dict(gate=dgate, up=dup, down=ddown, nw=dnw)
    norm = moe.moe_clip_grad_norm(list(grads.values()), max_norm)
    return dict(out=out, dwts=dwts, dx=dx, norm=norm, **grads)


@pytest.mark.parametrize("M,H,I,E,k,BS", [(150, 256, 128, 8, 2, 16), (1, 128, 64, 4, 2, 16), (700, 544, 288, 6, 3, 1),
                                          (64, 288, 96, 40, 2, 64)])
def test_training_step(moe, M, H, I, E, k, BS):
    log(f"4-bit training step M={M} H={H} I={I} E={E} top_k={k} BS={BS}")
    b = Block(M, H, I, E, M + H)
    r = Routed(moe, M, E, k, BS, M)
    got = train(moe, b, r, 1.0)
    torch.cuda.synchronize()

    # straight through: the values are those of the rounded weights, the gradients are theirs
    leaf = {n: mx_values(*mx_quantised(getattr(b, n))).requires_grad_() for n in ("gate", "up", "down")}
    leaf.update({n: getattr(b, n).double().requires_grad_() for n in ("res", "nw")})
    wts = r.weights.double().requires_grad_()
    z = b.x.double() + leaf["res"]
    n = z * (z.square().mean(1, keepdim=True) + EPS).pow(-0.5) * leaf["nw"]
    out = torch.zeros_like(z)
    for e in range(E):
        t, j = torch.nonzero(r.ids == e, as_tuple=True)
        if t.numel():
            v = n[t]
            h = torch.nn.functional.silu(v @ leaf["gate"][e].T) * (v @ leaf["up"][e].T)
            out = out.index_add(0, t, wts[t, j, None] * (h @ leaf["down"][e].T))
    total = (out * b.dout.double()).sum() + (z * b.dout.double()).sum()
    names = ["gate", "up", "down", "nw", "res"]
    ref = dict(zip(names + ["wts"], torch.autograd.grad(total, [leaf[x] for x in names] + [wts])))
    # hand-offs in bf16 as in the bf16 block: z, n, h, y, out; dy, dh, dz, dxs, dn, dx back
    close(got["out"], out.detach(), 5, "out")
    close(got["dwts"], ref["wts"], 5, "routing weights")
    close(got["dx"], ref["res"], 10, "input")
    # the norm of all gradients moves by no more than they do, and the clipped ones by both
    norm = math.sqrt(sum(float(ref[x].square().sum()) for x in ("gate", "up", "down", "nw")))
    assert abs(float(got["norm"]) - norm) <= 2 * 10 * STEP * norm
    for name, handoffs in (("down", 6), ("gate", 8), ("up", 8), ("nw", 10)):
        close(got[name], ref[name] * min(1.0, 1.0 / norm), handoffs + 10, name)


@pytest.mark.parametrize("M", [1, 77, 1000])
@pytest.mark.parametrize("H,I", [(512, 256), (288, 160)])
def test_serving_chain(moe, M, H, I):
    """Rows go to their experts in 4 bits and both products hand them on so; each stage is
    held to its own bounds on what the stage before handed over."""
    E, k = 8, 2
    g = gen(M + H)
    x, res, nw = randn(g, M, H), randn(g, M, H), randn(g, H, scale=0.1) + 1.0
    gate, up, down = mx_weight(g, E, I, H), mx_weight(g, E, I, H), mx_weight(g, E, H, I)
    r = Routed(moe, M, E, k, 16, M)
    n, _, _, _ = moe.moe_add_rms_norm(x, nw, EPS, residual=res)
    xs, xscale = moe.moe_mxfp4_quantize(n, r.perm, k, r.rows)
    h, hscale, _ = moe.moe_grouped_linear_mxfp4(xs, gate, r.offsets, r.counts, act="swiglu", up=up, x_scale=xscale, mxfp4_out=True)
    y, _, _ = moe.moe_grouped_linear_mxfp4(h, down, r.offsets, r.counts, x_scale=hscale)
    out = moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)
    torch.cuda.synchronize()

    p, kept = r.perm.long(), r.kept
    codes, scales = mx_quantised(n)
    assert torch.equal(mx_values(xs[p], xscale[p]), mx_values(codes, scales).repeat_interleave(k, 0))
    xv = torch.zeros(r.rows, H, dtype=torch.float64, device="cuda")
    xv[kept] = mx_values(xs[kept], xscale[kept])
    ref, err, _, _ = reference(r, xv, gate, up, None, None, None, "swiglu")
    check_mx_rows(h[kept], hscale[kept], ref[kept], err[kept], "gate+up")
    hv = torch.zeros(r.rows, I, dtype=torch.float64, device="cuda")
    hv[kept] = mx_values(h[kept], hscale[kept])
    ref, err, _, _ = reference(r, hv, down, None, None, None, None, "none")
    assert_within(y[kept], ref[kept], STEP * ref[kept].abs() + 2 * err[kept] + 1e-37, "down")
    rows = y[p].double().reshape(M, k, H) * r.weights.double()[..., None]
    assert_within(out, rows.sum(1), STEP * rows.sum(1).abs() + 4 * 2.0 ** -23 * rows.abs().sum(1) + 1e-37, "out")


def test_block_agrees_with_the_layer(moe):
    """Weights rounded here serve the layer kernels as they are, and give what the products
    give (which hand bf16 rows on, the layer float32 ones)."""
    M, H, I, E, k = 200, 256, 128, 8, 2
    g = gen(5)
    x = randn(g, M, H)
    gate, up, down = (moe.moe_mxfp4_quantize(randn(g, E, *s, scale=s[1] ** -0.5)) for s in ((I, H), (I, H), (H, I)))
    r = Routed(moe, M, E, k, 16, 5)
    xs, _ = moe.moe_permute(x, r.perm, k, r.rows)
    h, _, _ = moe.moe_grouped_linear_mxfp4(xs, gate, r.offsets, r.counts, act="swiglu", up=up)
    y, _, _ = moe.moe_grouped_linear_mxfp4(h, down, r.offsets, r.counts)
    out = moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)
    ref = moe.MoeLayer(gate, up, down, k, 16).forward(x, r.ids, r.weights)
    torch.cuda.synchronize()
    close(out, ref, 4, "layer")  # h, y and both outputs


def test_training_step_in_a_graph(moe):
    """One captured step replays for new rows, weights and routings, eager steps and
    synchronizations between the replays."""
    M, H, I, E, k = 300, 288, 160, 8, 2
    b, r = Block(M, H, I, E, 1), Routed(moe, M, E, k, 16, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        train(moe, b, r, 1.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = train(moe, b, r, 1.0)
    for seed in (5, 6, 7):
        other, route = Block(M, H, I, E, seed), Routed(moe, M, E, k, 16, seed)
        for n, v in vars(b).items():
            v.copy_(getattr(other, n))
        for n in ("offsets", "counts", "perm", "weights"):
            getattr(r, n).copy_(getattr(route, n))
        graph.replay()
        torch.cuda.synchronize()
        # rows outside the runs belong to no result, so every result is compared whole
        got = {n: v.clone() for n, v in outs.items()}
        for n, v in train(moe, b, r, 1.0).items():
            assert torch.equal(got[n], v), n


def test_serving_in_a_graph(moe):
    M, H, I, E, k = 40, 256, 128, 8, 2
    g = gen(3)
    gate, up, down = mx_weight(g, E, I, H), mx_weight(g, E, I, H), mx_weight(g, E, H, I)
    x, r = randn(g, M, H), Routed(moe, M, E, k, 16, 2)

    def serve():
        xs, xscale = moe.moe_mxfp4_quantize(x, r.perm, k, r.rows)
        h, hscale, _ = moe.moe_grouped_linear_mxfp4(xs, gate, r.offsets, r.counts, act="swiglu", up=up, x_scale=xscale, mxfp4_out=True)
        y, _, _ = moe.moe_grouped_linear_mxfp4(h, down, r.offsets, r.counts, x_scale=hscale)
        return moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        serve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = serve()
    for seed in (11, 12, 13):
        x.copy_(randn(gen(seed), M, H))
        route = Routed(moe, M, E, k, 16, seed)
        for n in ("offsets", "counts", "perm", "weights"):
            getattr(r, n).copy_(getattr(route, n))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, serve())


def test_two_streams_at_once(moe):
    """Two steps on two streams share nothing."""
    blocks = [(Block(400, 256, 128, 8, s), Routed(moe, 400, 8, 2, 16, s)) for s in (1, 2)]
    want = [train(moe, b, r, 1.0) for b, r in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        got = []
        for (b, r), st in zip(blocks, streams):
            with torch.cuda.stream(st):
                got.append(train(moe, b, r, 1.0))
        torch.cuda.synchronize()
        for a, c in zip(want, got):
            for n in a:
                assert torch.equal(a[n], c[n]), n


def test_a_row_has_the_same_bits_in_any_series_of_tiles(moe):
    """A workgroup's tiles run one after another: the rows of a tile give what they give
    alone, and every call gives the same bits."""
    E, N, K = 24, 544, 672
    g = gen(17)
    counts = torch.randint(0, 300, (E,), generator=g, device="cuda", dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    rows = int(offsets[-1])
    x = randn(g, rows, K)
    w, up = mx_weight(g, E, N, K), mx_weight(g, E, N, K)
    q, s = moe.moe_mxfp4_quantize(x)
    for a, xs in ((x, None), (q, s)):
        y, _, pre = moe.moe_grouped_linear_mxfp4(a, w, offsets, counts, act="swiglu", up=up, x_scale=xs, save_preact=True)
        for _ in range(3):
            again, _, pre2 = moe.moe_grouped_linear_mxfp4(a, w, offsets, counts, act="swiglu", up=up, x_scale=xs, save_preact=True)
            assert torch.equal(y, again) and torch.equal(pre, pre2)
    dz = randn(g, rows, 2 * N)
    dx = moe.moe_grouped_linear_mxfp4_backward_x(dz, w, offsets, counts, up=up)
    assert all(torch.equal(dx, moe.moe_grouped_linear_mxfp4_backward_x(dz, w, offsets, counts, up=up)) for _ in range(3))


def test_binding_refuses_mismatches(moe):
    """Shapes, types and strides that do not fit are refused before a launch."""
    bf, u8 = torch.bfloat16, torch.uint8
    x = torch.zeros(4, 256, dtype=bf, device="cuda")
    c, s = torch.zeros(4, 128, dtype=u8, device="cuda"), torch.zeros(4, 8, dtype=u8, device="cuda")
    w = (torch.zeros(3, 64, 128, dtype=u8, device="cuda"), torch.zeros(3, 64, 8, dtype=u8, device="cuda"))
    off, cnt = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    perm = torch.zeros(8, dtype=torch.int32, device="cuda")
    calls = [
        lambda: moe.moe_mxfp4_quantize(x[:, :40]), lambda: moe.moe_mxfp4_quantize(x[:, ::2]), lambda: moe.moe_mxfp4_quantize(x.half()),
        lambda: moe.moe_mxfp4_quantize(x, perm, 3, 8), lambda: moe.moe_mxfp4_quantize(x, perm, 2), lambda: moe.moe_mxfp4_quantize(x, None, 2, 8),
        lambda: moe.moe_mxfp4_quantize(x, perm.long(), 2, 8), lambda: moe.moe_mxfp4_quantize(x, codes=c[:3]),
        lambda: moe.moe_mxfp4_quantize(x, scales=s.float()), lambda: moe.moe_mxfp4_quantize(x.view(2, 2, 256).transpose(0, 1)),
        lambda: moe.moe_mxfp4_dequantize(c, s[:3].contiguous()), lambda: moe.moe_mxfp4_dequantize(c[:, :100].contiguous(), s),
        lambda: moe.moe_mxfp4_dequantize(c.view(torch.int8), s), lambda: moe.moe_mxfp4_dequantize(c, s, dtype=torch.float16),
        lambda: moe.moe_grouped_linear_mxfp4(x, w), lambda: moe.moe_grouped_linear_mxfp4(x, w[0], off, cnt),
        lambda: moe.moe_grouped_linear_mxfp4(x, (w[0], w[1].float()), off, cnt), lambda: moe.moe_grouped_linear_mxfp4(c, w, off, cnt),
        lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, x_scale=s), lambda: moe.moe_grouped_linear_mxfp4(c, w, off, cnt, x_scale=s[:, :4].contiguous()),
        lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, act="swiglu"), lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, up=w),
        lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt[:2].contiguous()), lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, out_scale=s),
        lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, bias=x[0]), lambda: moe.moe_grouped_linear_mxfp4(x, w, off, cnt, residual=x),
        lambda: moe.moe_grouped_linear_mxfp4(x, (w[0][:, :40].contiguous(), w[1][:, :40].contiguous()), off, cnt, mxfp4_out=True),
        lambda: moe.moe_grouped_linear_mxfp4_backward_x(x, w, off, cnt), lambda: moe.moe_grouped_linear_mxfp4_backward_x(x.float(), w, off, cnt),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
            log(f"call {i} was not refused")


def test_readme_block(moe):
    """README's 4-bit block as it is printed: it runs, its two chains agree with the calls
    on the values they stand for, and the gradients' norm is theirs."""
    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(readme).read(), flags=re.S) if "moe_clip_grad_norm" in b]
    assert len(blocks) == 1
    M, H, I, E, k = 90, 128, 96, 6, 2
    log("README 4-bit block")
    b = Block(M, H, I, E, 5)
    r = Routed(moe, M, E, k, 16, 5)
    g = gen(6)
    grads = {n: randn(g, E, I, H) for n in ("dgate", "dup")} | {"ddown": randn(g, E, H, I), "dnorm_w": randn(g, H)}
    before = {n: t.clone() for n, t in grads.items()}
    x_rows, _ = moe.moe_permute(b.x, r.perm, k, r.rows)
    got = dict(grads, moe=moe, gate=b.gate, up=b.up, down=b.down, n=b.x, perm=r.perm, k=k, rows=r.rows, off=r.offsets, cnt=r.counts,
               x_rows=x_rows, dz=randn(g, r.rows, 2 * I))
    exec(blocks[0], got)
    torch.cuda.synchronize()
    kept = r.kept
    assert torch.equal(got["xs"][kept], moe.moe_mxfp4_quantize(x_rows)[0][kept])
    h, _, pre = moe.moe_grouped_linear_mxfp4(x_rows, got["gate4"], r.offsets, r.counts, act="swiglu", up=got["up4"], save_preact=True)
    assert torch.equal(got["h"][kept], h[kept]) and torch.equal(got["pre"][kept], pre[kept])
    assert got["y"].shape == (r.rows, H) and got["dx_rows"].shape == (r.rows, H) and bool(got["y"][kept].isfinite().all())
    norm = sum(float(t.double().square().sum()) for t in before.values()) ** 0.5
    assert abs(float(got["norm"]) - norm) <= norm * 2.0 ** -23
    for n, t in grads.items():
        assert_within(t, before[n].double() / norm, (STEP + 2.0 ** -22) * before[n].double().abs() / norm)
