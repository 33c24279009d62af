"""The operators together, as an expert block uses them: a training step in bf16
against float64 autograd, the 8-bit serving chain, and both beside the layer
kernels this library serves the same experts with."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import Routed, assert_within, check_fp8_rows, dequantised, gen, half, randn

pytestmark = pytest.mark.gpu

EPS = 1e-6
STEP = half(torch.bfloat16)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


def close(got, ref, handoffs, what):
    """2-norm distance: each of `handoffs` roundings to bf16 on the way moves every
    value by at most half a step, 2^-8 of it; the products keep independent relative
    errors at their size, and a factor 2 covers the sums that cancel."""
    got, ref = got.double(), ref.double()
    off = float((got - ref).norm() / ref.norm())
    assert off <= 2 * handoffs * STEP, (what, off, 2 * handoffs * STEP)


class Block:
    def __init__(self, moe, M, H, I, E, k, seed):
        g = gen(seed)
        self.x, self.res = randn(g, M, H), randn(g, M, H)
        self.nw = randn(g, H, scale=0.1) + 1.0
        self.gate, self.up = randn(g, E, I, H, scale=H ** -0.5), randn(g, E, I, H, scale=H ** -0.5)
        self.down = randn(g, E, H, I, scale=I ** -0.5)
        self.rw = randn(g, E, H, scale=H ** -0.5)
        self.dout = randn(g, M, H)


def forward(moe, b, k, BS):
    M, H = b.x.shape
    E = b.gate.shape[0]
    n, _, z, rstd = moe.moe_add_rms_norm(b.x, b.nw, EPS, residual=b.res, save_rstd=True)
    ids, wts, _ = moe.moe_router_topk(n, b.rw, k)
    t = moe.moe_align(ids, E, BS)
    rows = t.sorted_token_ids.numel()
    off, cnt, perm = t.expert_offsets, t.expert_counts, t.token_to_perm
    xs, _ = moe.moe_permute(n, perm, k, rows)
    h, _, pre = moe.moe_grouped_linear(xs, b.gate, off, cnt, act="swiglu", up=b.up, save_preact=True)
    y, _, _ = moe.moe_grouped_linear(h, b.down, off, cnt)
    out = moe.moe_unpermute(y, perm, k, topk_weights=wts)
    return dict(n=n, z=z, rstd=rstd, ids=ids, wts=wts, perm=perm, off=off, cnt=cnt, xs=xs, h=h, pre=pre, y=y, out=out)


def backward(moe, b, s, k):
    dy, dwts = moe.moe_unpermute_backward(b.dout, s["y"], s["perm"], s["wts"])
    dh = moe.moe_grouped_linear_backward_x(dy, b.down, s["off"], s["cnt"])
    ddown, _, _, _ = moe.moe_grouped_linear_backward_w(dy, s["h"], s["off"], s["cnt"])
    dz = moe.moe_grouped_act_backward(dh, s["pre"], "swiglu", s["off"], s["cnt"])
    dxs = moe.moe_grouped_linear_backward_x(dz, b.gate, s["off"], s["cnt"], up=b.up)
    dgate, dup, _, _ = moe.moe_grouped_linear_backward_w(dz, s["xs"], s["off"], s["cnt"], gated=True)
    dn = moe.moe_unpermute(dxs, s["perm"], k)
    dx, dnw = moe.moe_add_rms_norm_backward(dn, s["z"], b.nw, s["rstd"], dz=b.dout)  # the stream's own gradient
    return dict(dwts=dwts, ddown=ddown, dgate=dgate, dup=dup, dx=dx, dnw=dnw)


@pytest.mark.parametrize("M,H,I,E,k,BS", [(150, 256, 128, 8, 2, 16), (1, 128, 64, 4, 2, 16), (700, 520, 264, 6, 3, 1),
                                          (64, 264, 72, 40, 2, 64)])
def test_training_step(moe, M, H, I, E, k, BS):
    log(f"training step M={M} H={H} I={I} E={E} top_k={k} BS={BS}")
    b = Block(moe, M, H, I, E, k, M + H)
    s = forward(moe, b, k, BS)
    grads = backward(moe, b, s, k)
    torch.cuda.synchronize()

    leaf = {n: getattr(b, n).double().requires_grad_() for n in ("res", "nw", "gate", "up", "down")}
    wts = s["wts"].double().requires_grad_()
    z = b.x.double() + leaf["res"]
    n = z * (z.square().mean(1, keepdim=True) + EPS).pow(-0.5) * leaf["nw"]
    out = torch.zeros_like(z)
    for e in range(E):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        v = n[t]
        h = torch.nn.functional.silu(v @ leaf["gate"][e].T) * (v @ leaf["up"][e].T)
        out = out.index_add(0, t, wts[t, j, None] * (h @ leaf["down"][e].T))
    total = (out * b.dout.double()).sum() + (z * b.dout.double()).sum()  # the block's output and the stream both go on
    names = ["res", "nw", "gate", "up", "down"]
    g = torch.autograd.grad(total, [leaf[x] for x in names] + [wts])
    # z, n, h, y, out
    close(s["out"], out.detach(), 5, "out")
    # forward hand-offs and dy, dh, dz, dxs, dn, dx on the way back
    close(grads["dwts"], g[5], 5, "routing weights")
    close(grads["ddown"], g[4], 6, "down")
    close(grads["dgate"], g[2], 8, "gate")
    close(grads["dup"], g[3], 8, "up")
    close(grads["dx"], g[0], 10, "input")
    close(grads["dnw"], g[1], 10, "norm weight")


def test_block_agrees_with_the_layer(moe):
    """The same experts through the layer kernels (float32 intermediates)."""
    b = Block(moe, 200, 256, 128, 8, 2, 3)
    s = forward(moe, b, 2, 16)
    layer = moe.MoeLayer((b.gate, None), (b.up, None), (b.down, None), 2, 16)
    ref = layer.forward(s["n"], s["ids"], s["wts"])
    torch.cuda.synchronize()
    close(s["out"], ref, 4, "layer")  # h, y and both outputs


@pytest.mark.parametrize("M", [1, 77, 1000])
def test_8bit_serving_chain(moe, M):
    """Norm, permutation and both products hand 8-bit rows on; each stage is held to
    its own bounds on what the stage before handed over."""
    H, I, E, k = 512, 256, 8, 2
    g = gen(M)
    x, res, nw = randn(g, M, H), randn(g, M, H), randn(g, H, scale=0.1) + 1.0

    def weight(N, K):
        v = torch.randn(E, N // 128, 128, K // 128, 128, generator=g, device="cuda") * K ** -0.5
        sc = v.abs().amax((2, 4)) / 448
        return (v / sc[:, :, None, :, None]).to(torch.float8_e4m3fn).reshape(E, N, K).view(torch.uint8), sc.contiguous()

    gate, up, down = weight(I, H), weight(I, H), weight(H, I)
    r = Routed(moe, M, E, k, 16, M)
    codes, scale, z, _ = moe.moe_add_rms_norm(x, nw, EPS, residual=res, fp8=True)
    xs, xscale = moe.moe_permute(codes, r.perm, k, r.rows, scale=scale)
    h, hscale, _ = moe.moe_grouped_linear(xs, gate, r.offsets, r.counts, act="swiglu", up=up, x_scale=xscale, fp8_out=True)
    y, _, _ = moe.moe_grouped_linear(h, down, r.offsets, r.counts, x_scale=hscale)
    out = moe.moe_unpermute(y, r.perm, k, topk_weights=r.weights)
    torch.cuda.synchronize()

    n = z.double() * (z.double().square().mean(1, keepdim=True) + EPS).pow(-0.5) * nw.double()
    check_fp8_rows(codes, scale, n, n.abs() * 2.0 ** -18, "norm")

    def w64(w, e):
        return w[0][e].view(torch.float8_e4m3fn).double() * w[1][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)

    p = r.perm.long()
    assert torch.equal(xs.view(torch.uint8)[p], codes.view(torch.uint8).repeat_interleave(k, 0))
    for e, at, c in r.runs:
        if c == 0:
            continue
        s = slice(at, at + c)
        v, m = dequantised(xs.view(torch.uint8)[s], xscale[s]), 2.0 ** -23
        zg, zu = v @ w64(gate, e).T, v @ w64(up, e).T
        ge, ue = (H + 8) * m * (v.abs() @ w64(gate, e).abs().T), (H + 8) * m * (v.abs() @ w64(up, e).abs().T)
        a = zg * torch.sigmoid(zg)
        err = 1.13 * ge * (zu.abs() + ue) + a.abs() * ue + 16 * m * (a * zu).abs()
        check_fp8_rows(h.view(torch.uint8)[s], hscale[s], a * zu, err, "gate+up")
        v = dequantised(h.view(torch.uint8)[s], hscale[s])
        ref, mag = v @ w64(down, e).T, v.abs() @ w64(down, e).abs().T
        assert_within(y[s], ref, STEP * ref.abs() + 2 * (I + 8) * m * mag + 1e-37, "down")
    rows = y[p].double().reshape(M, k, H) * r.weights.double()[..., None]
    assert_within(out, rows.sum(1), STEP * rows.sum(1).abs() + 4 * 2.0 ** -23 * rows.abs().sum(1) + 1e-37, "out")


def test_training_step_in_a_graph(moe):
    """One captured step replays for new inputs and routings, eager steps and
    synchronizations between the replays."""
    M, H, I, E, k, BS = 300, 264, 136, 8, 2, 16
    b = Block(moe, M, H, I, E, k, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    keys = ("out", "wts")

    def step():
        s = forward(moe, b, k, BS)
        return {**{n: s[n] for n in keys}, **backward(moe, b, s, k)}

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    for seed in (5, 6, 7):
        g = gen(seed)
        b.x.copy_(randn(g, M, H))
        b.dout.copy_(randn(g, M, H))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in outs.items()}
        for n, v in step().items():
            assert torch.equal(got[n], v), n


def test_two_streams_at_once(moe):
    """Two steps on two streams share nothing."""
    blocks = [Block(moe, 400, 256, 128, 8, 2, s) for s in (1, 2)]
    want = []
    for b in blocks:
        s = forward(moe, b, 2, 16)
        want.append((s["out"], backward(moe, b, s, 2)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = []
    for _ in range(3):
        got.clear()
        for b, st in zip(blocks, streams):
            with torch.cuda.stream(st):
                s = forward(moe, b, 2, 16)
                got.append((s["out"], backward(moe, b, s, 2)))
        torch.cuda.synchronize()
        for (o, d), (oo, dd) in zip(want, got):
            assert torch.equal(o, oo)
            for n in d:
                assert torch.equal(d[n], dd[n]), n


def test_binding_refuses_mismatches(moe):
    """Shapes, types and strides that do not fit are refused before a launch."""
    bf = torch.bfloat16
    x, w = torch.zeros(4, 256, dtype=bf, device="cuda"), torch.ones(256, dtype=bf, device="cuda")
    perm, wts = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.ones(4, 2, device="cuda")
    E3 = torch.zeros(3, 64, 256, dtype=bf, device="cuda")
    off, cnt = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    f8 = torch.zeros(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    calls = [
        lambda: moe.moe_add_rms_norm(x, w[:128].contiguous(), EPS),
        lambda: moe.moe_add_rms_norm(x, w, EPS, residual=x[:2]),
        lambda: moe.moe_add_rms_norm(x[:, ::2], w[:128].contiguous(), EPS),
        lambda: moe.moe_add_rms_norm(x, w, EPS, residual_out=x),
        lambda: moe.moe_add_rms_norm(x[:, :200], w[:200].contiguous(), EPS, fp8=True),
        lambda: moe.moe_add_rms_norm(x, w, EPS, out=x.float()),
        lambda: moe.moe_add_rms_norm_backward(x, x.float(), w, wts[:, 0].contiguous(), dz=x),
        lambda: moe.moe_permute(x, perm, 3, 8),
        lambda: moe.moe_permute(f8, perm, 2, 8),
        lambda: moe.moe_permute(x, perm.long(), 2, 8),
        lambda: moe.moe_unpermute(x, perm, 2, topk_weights=wts.double()),
        lambda: moe.moe_unpermute_backward(x[:3].contiguous(), x, perm, wts),
        lambda: moe.moe_grouped_linear(x, E3),
        lambda: moe.moe_grouped_linear(x, E3, off, None),
        lambda: moe.moe_grouped_linear(x, E3, off, cnt[:2].contiguous()),
        lambda: moe.moe_grouped_linear(x, E3, off, cnt, act="swiglu"),
        lambda: moe.moe_grouped_linear(x, E3, off, cnt, up=E3),
        lambda: moe.moe_grouped_linear(x, E3, off, cnt, bias=w),
        lambda: moe.moe_grouped_linear(x, E3, off, cnt, fp8_out=True),
        lambda: moe.moe_grouped_linear(f8, E3, off, cnt),
        lambda: moe.moe_grouped_linear(x, (E3.view(torch.uint8), None), off, cnt),
        lambda: moe.moe_grouped_linear_backward_x(x, E3, off, cnt),
        lambda: moe.moe_grouped_linear_backward_w(x, x[:2].contiguous(), off, cnt),
        lambda: moe.moe_grouped_linear_backward_w(x, x, off, cnt, dtype=torch.float16),
        lambda: moe.moe_grouped_act_backward(x, x, "swiglu"),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
            log(f"call {i} was not refused")
