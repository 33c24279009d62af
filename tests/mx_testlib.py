"""MXFP4 helpers for the tests of the 4-bit operators: the format from its definition in
float64, and the products' reference values with bounds that count every rounding."""

from __future__ import annotations

import torch

from ops_testlib import SUM, assert_within, randn
from test_gpu_ops_linear import ACT, SLOPE, act64

MX = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def power(byte):
    """2^(byte - 127) in float64, exactly (the device's pow is off by a unit in the last
    place for some exponents); NaN for 255."""
    t = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [float("nan")], dtype=torch.float64, device=byte.device)
    return t[byte.long()]


def mx_bytes(amax):
    """Scale bytes of blocks with these absolute maxima (float64)."""
    e = torch.frexp(amax).exponent - 1  # amax in [2^e, 2^(e+1))
    byte = torch.clamp(e - 2 + 127, min=2)
    byte = torch.where(amax == 0, torch.full_like(byte, 127), byte)
    return torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255))


def mx_quantised(v):
    """(codes without a sign on zeros, scale bytes) of rows, by search among the magnitudes."""
    b = v.double().reshape(*v.shape[:-1], -1, MX)
    byte = mx_bytes(b.abs().amax(-1))
    m = torch.where(byte[..., None] == 255, 0.0, b.abs() / power(byte)[..., None])
    best, dist = torch.zeros_like(m, dtype=torch.int64), m.clone()
    for c in range(1, 8):
        d = (m - MAGNITUDES[c]).abs()
        take = (d < dist) | ((d == dist) & (c % 2 == 0))
        best, dist = torch.where(take, c, best), torch.where(take, d, dist)
    best = torch.where((b < 0) & (best > 0), best + 8, best).reshape(v.shape)
    return (best[..., 0::2] | best[..., 1::2] << 4).to(torch.uint8), byte.to(torch.uint8)


def unsigned_zeros(codes):
    """Packed codes with -0 as 0."""
    lo, hi = codes & 15, codes >> 4
    return torch.where(lo == 8, 0, lo) | torch.where(hi == 8, 0, hi) << 4


def mx_values(codes, scales):
    """float64 values of packed codes and scale bytes."""
    t = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64, device=codes.device)
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).reshape(*codes.shape[:-1], -1)
    return v * power(scales).repeat_interleave(MX, -1)


def mx_weight(g, E, N, K):
    return mx_quantised(torch.randn(E, N, K, generator=g, device="cuda") * K ** -0.5)


def mx_rows(g, rows, K):
    return mx_quantised(randn(g, rows, K))


def reference(r, x, w, up, bias, up_bias, residual, act):
    """y, its error bound before the last rounding, and the pre-activations with theirs;
    x float64 [rows, K], w and up MXFP4 pairs."""
    N = w[0].shape[1]
    wide = 1 if up is None else 2
    y = torch.zeros(r.rows, N, dtype=torch.float64, device="cuda")
    yerr, pre = torch.zeros_like(y), torch.zeros(r.rows, wide * N, dtype=torch.float64, device="cuda")
    perr = torch.zeros_like(pre)
    for e, at, n in r.runs:
        if n == 0:
            continue
        s = slice(at, at + n)

        def product(weights, b):
            m = mx_values(weights[0][e], weights[1][e])
            z, mag = x[s] @ m.T, x[s].abs() @ m.abs().T
            if b is not None:
                z, mag = z + b[e].double(), mag + b[e].double().abs()
            return z, (x.shape[1] + 8) * SUM * mag

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


def check_mx_rows(codes, scales, y, yerr, what=""):
    """MXFP4 rows against float64 rows y known to yerr: each byte is that of a maximum
    within its error, each value within half a step of y cut off at 6 scales (steps are
    half of the scale below 2 scales, above at most half of the value)."""
    if y.shape[0] == 0:
        return
    b, e = y.reshape(y.shape[0], -1, MX).abs(), yerr.reshape(y.shape[0], -1, MX)
    lo, hi = mx_bytes((b - e).clamp(min=0).amax(-1)), mx_bytes((b + e).amax(-1))
    got = scales.long()
    # a maximum that may round to zero may also make a block of zeros
    ok = ((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi)))
    assert bool(ok.all()), (what + " scale bytes", int((~ok).sum()))
    s = power(scales).repeat_interleave(MX, -1)
    cut = torch.minimum(torch.maximum(y, -6 * s), 6 * s)
    assert_within(mx_values(codes, scales), cut, torch.maximum(cut.abs() / 4, s / 4) + yerr, what + " codes")
