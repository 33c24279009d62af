"""Helpers shared by the tests of the operators around the layer: seeded rows,
alignment tables from the library's own align, and error bounds.

Expected values are computed in float64 from the formulas, on the same bf16 or
e4m3 inputs.  Bounds count every rounding: a result rounded to type t is off by at
most ``half(t)`` relative to its value, and a float32 sum of n products by at most
``n * 2^-23`` times the sum of their absolute values (twice the worst case of a
sequential sum with products rounded; the matrix cores' order is not specified).
"""

from __future__ import annotations

import math

import torch

BLOCK = 128
SUM = 2.0 ** -23


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def assert_within(got, ref, bound, what=""):
    """|got - ref| <= bound everywhere (all float64), NaN nowhere."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.numel() == 0:
        return
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), float((err / bound).nan_to_num(math.inf).max()))


def quantised(v):
    """Rows as e4m3fn codes and scales per 128 columns (torch's rounding)."""
    b = v.float().reshape(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    scale = torch.where(amax > 0, torch.clamp(amax / 448, min=2.0 ** -126), torch.ones_like(amax))
    return (b / scale[..., None]).to(torch.float8_e4m3fn).reshape(v.shape), scale


def dequantised(codes, scale):
    """float64 values of 8-bit rows."""
    if codes.dtype == torch.uint8:
        codes = codes.view(torch.float8_e4m3fn)
    return codes.double() * scale.double().repeat_interleave(BLOCK, 1)


def check_fp8_rows(codes, scale, y, yerr, what=""):
    """8-bit rows against float64 rows y known to yerr: every scale is the block
    maximum over 448, every value within half a step (2^-4 relative, half of the
    smallest subnormal 2^-9 at the low end, both times the scale)."""
    if y.shape[0] == 0:
        return
    b, e = y.reshape(y.shape[0], -1, BLOCK), yerr.reshape(y.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    ref = torch.where(amax > 0, torch.clamp(amax / 448, min=2.0 ** -126), torch.ones_like(amax))
    # a division rounds once more
    assert_within(scale, ref, e.amax(-1) / 448 + ref * 2.0 ** -23, what + " scale")
    s = scale.double()[..., None].expand_as(b).reshape(y.shape)
    bound = 2.0 ** -4 * (y.abs() + yerr) + s * 2.0 ** -10 + yerr + y.abs() * 2.0 ** -22
    assert_within(dequantised(codes, scale), y, bound, what + " codes")


class Routed:
    """Slots over experts, aligned by the library.  `mode`: "random", "one" (every
    slot on expert 0), "skew" (most slots on a few), with a part dropped."""

    def __init__(self, moe, M, E, k, BS, seed, mode="random", drop=0.0):
        g = gen(seed)
        self.M, self.E, self.k, self.BS = M, E, k, BS
        if mode == "one":
            ids = torch.zeros(M, k, dtype=torch.int64, device="cuda")
        else:
            bias = 4.0 * torch.randn(E, generator=g, device="cuda") if mode == "skew" else 0.0
            logits = torch.randn(M, E, generator=g, device="cuda") + bias
            ids = torch.topk(logits, k, dim=1).indices
        if drop:
            ids = torch.where(torch.rand(M, k, generator=g, device="cuda") < drop, -1, ids)
        self.ids = ids.contiguous()
        self.weights = torch.rand(M, k, generator=g, device="cuda") + 0.1
        self.t = moe.moe_align(self.ids, E, BS)
        torch.cuda.synchronize()
        self.rows = self.t.sorted_token_ids.numel()
        self.offsets, self.counts, self.perm = self.t.expert_offsets, self.t.expert_counts, self.t.token_to_perm
        off, cnt = self.offsets.tolist(), self.counts.tolist()
        self.runs = [(e, off[e], cnt[e]) for e in range(E)]
        self.kept = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for _, at, n in self.runs:
            self.kept[at:at + n] = True


class Dense:
    """One expert that holds every row."""

    def __init__(self, rows):
        self.rows, self.E, self.offsets, self.counts = rows, 1, None, None
        self.runs = [(0, 0, rows)]
        self.kept = torch.ones(rows, dtype=torch.bool, device="cuda")


def poison(t, kept):
    """Rows outside every run become NaN: nothing may read them into a result."""
    if t.dtype == torch.float8_e4m3fn:
        t.view(torch.uint8)[~kept] = 0x7F
    else:
        t[~kept] = float("nan")
    return t


SENTINEL = 0x5A


def untouched_buffer(*shape, dtype):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(SENTINEL)
    return t


def assert_untouched(t, kept, what=""):
    rest = t[~kept].contiguous().view(torch.uint8) if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8)[~kept]
    assert bool((rest == SENTINEL).all()), f"{what}: rows outside every run were written"
