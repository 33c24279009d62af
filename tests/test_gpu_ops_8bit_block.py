"""A block with 8-bit rows and its router: the norm's bf16 rows go to the router, its
8-bit rows of the same stream to the experts."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import BLOCK, SUM, check_fp8_rows, dequantised, gen, half, randn

pytestmark = pytest.mark.gpu

EPS = 1e-6


def weight(g, E, N, K):
    v = torch.randn(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK, generator=g, device="cuda") * K ** -0.5
    sc = v.abs().amax((2, 4)) / 448
    return (v / sc[:, :, None, :, None]).to(torch.float8_e4m3fn).reshape(E, N, K).view(torch.uint8), sc.contiguous()


def w64(w, e):
    return w[0][e].view(torch.float8_e4m3fn).double() * w[1][e].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


@pytest.mark.parametrize("M,stream", [(1, torch.bfloat16), (90, torch.float32), (1000, torch.bfloat16)])
def test_block_with_router(M, stream):
    import mixture_experts_routing_align_amd as moe

    log(f"8-bit block M={M} {stream}")
    H, I, E, k, BS = 512, 256, 16, 4, 16
    g = gen(M)
    x, res, nw = randn(g, M, H), randn(g, M, H, dtype=stream), randn(g, H, scale=0.1) + 1.0
    rw = randn(g, E, H, scale=H ** -0.5)
    gate, up, down = weight(g, E, I, H), weight(g, E, I, H), weight(g, E, H, I)
    z64 = (x.float() + res.float()).to(stream).double()

    n, _, z, rstd = moe.moe_add_rms_norm(x, nw, EPS, residual=res, save_rstd=True)
    codes, scale, z8, rstd8 = moe.moe_add_rms_norm(x, nw, EPS, residual=res, fp8=True, save_rstd=True, residual_out=res)
    ids, wts, _ = moe.moe_router_topk(n, rw, k)
    t = moe.moe_align(ids, E, BS)
    off, cnt, perm = t.expert_offsets, t.expert_counts, t.token_to_perm
    xs, xscale = moe.moe_permute(codes, perm, k, t.sorted_token_ids.numel(), scale=scale)
    h, hscale, _ = moe.moe_grouped_linear(xs, gate, off, cnt, act="swiglu", up=up, x_scale=xscale, fp8_out=True)
    y, _, _ = moe.moe_grouped_linear(h, down, off, cnt, x_scale=hscale)
    out = moe.moe_unpermute(y, perm, k, topk_weights=wts)
    torch.cuda.synchronize()

    # one stream, one rstd, two roundings of one y
    assert z8.data_ptr() == res.data_ptr() and torch.equal(z, z8) and torch.equal(z.double(), z64) and torch.equal(rstd, rstd8)
    n64 = z64 * rstd.double()[:, None] * nw.double()
    assert bool(((n.double() - n64).abs() <= half(torch.bfloat16) * n64.abs() + 4 * SUM * n64.abs()).all())
    check_fp8_rows(codes, scale, n64, 4 * SUM * n64.abs(), "norm")

    a, ref = dequantised(codes, scale), torch.zeros(M, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        at, j = torch.nonzero(ids == e, as_tuple=True)
        v = a[at]
        m = torch.nn.functional.silu(v @ w64(gate, e).T) * (v @ w64(up, e).T)
        ref = ref.index_add(0, at, wts[at, j, None].double() * (m @ w64(down, e).T))
    # h is rounded to 8 bits, y and out to bf16; a factor 2 covers sums that cancel
    off = float((out.double() - ref).norm() / ref.norm())
    assert off <= 2 * (half(torch.float8_e4m3fn) + 2 * half(torch.bfloat16)), off
