"""The operators' C ABI on the host: every declared symbol is exported, the sizing
functions answer, and every host-side check refuses bad arguments before touching
the GPU (no compute call runs here)."""

import ctypes
import os
import re

import pytest
import torch

import mixture_experts_routing_align_amd as moe
from mixture_experts_routing_align_amd import _ffi

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x_ops.h")
A = 0x1000   # non-NULL aligned address no call may dereference: every case fails before any launch
ODD = 0x1008
OK, NULL, SHAPE, LIMIT, WS = (_ffi.MOE_OK, _ffi.MOE_ERR_NULL, _ffi.MOE_ERR_SHAPE, _ffi.MOE_ERR_LIMIT, _ffi.MOE_ERR_WORKSPACE)
BF16, F32, E4M3 = _ffi.MOE_DT_BF16, _ffi.MOE_DT_F32, _ffi.MOE_DT_E4M3


@pytest.fixture(scope="module")
def lib():
    return _ffi.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(_ffi.OPS_SIGNATURES)
    for name in names:
        assert hasattr(lib, name), name
    assert lib.moe_ops_abi_version() == 1


def test_descriptor_layout():
    """The ctypes descriptor has the C struct's size: 8 + 3*4 + 3*4 + 2 pointers,
    x, x_scale, two weight pairs and six more pointers."""
    assert ctypes.sizeof(_ffi.MoeLinearDesc) == 8 + 12 + 12 + 14 * 8


def norm(lib, x=A, ldx=256, res=None, rdt=BF16, res_out=None, w=A, eps=1e-6, out=A, odt=BF16, scale=None, rstd=None, M=4, H=256):
    return lib.moe_add_rms_norm(x, ldx, res, rdt, res_out, w, eps, out, odt, scale, rstd, M, H, None)


def test_norm_refusals(lib):
    assert norm(lib, M=0, x=None, w=None, out=None) == OK
    assert norm(lib, M=-1) == SHAPE
    assert norm(lib, M=2 ** 31) == LIMIT
    assert norm(lib, H=0) == SHAPE
    assert norm(lib, H=_ffi.MOE_NORM_MAX_H + 1, ldx=2 ** 20) == LIMIT
    assert norm(lib, ldx=255) == SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == SHAPE
    assert norm(lib, res=A, rdt=E4M3) == SHAPE
    assert norm(lib, res_out=A) == SHAPE
    assert norm(lib, odt=F32) == SHAPE
    assert norm(lib, odt=E4M3, H=200, ldx=200) == SHAPE
    assert norm(lib, odt=E4M3) == NULL  # no scales
    assert norm(lib, x=None) == NULL
    assert norm(lib, w=None) == NULL
    assert norm(lib, out=None) == NULL
    assert "out" in lib.moe_last_error().decode()


def norm_backward(lib, dy=A, z=A, zdt=BF16, w=A, rstd=A, dz=None, dx=A, dw=A, M=4000, H=256, ws=A, ws_bytes=1 << 30):
    return lib.moe_add_rms_norm_backward(dy, z, zdt, w, rstd, dz, dx, dw, M, H, ws, ws_bytes, None)


def test_norm_backward_refusals(lib):
    need = lib.moe_add_rms_norm_backward_workspace_bytes(4000, 256)
    assert need > 0 and need % (256 * 4) == 0
    assert lib.moe_add_rms_norm_backward_workspace_bytes(1, 256) == 0
    assert lib.moe_add_rms_norm_backward_workspace_bytes(0, 256) == 0
    assert lib.moe_add_rms_norm_backward_workspace_bytes(-1, 256) == 0
    assert lib.moe_add_rms_norm_backward_workspace_bytes(4000, 0) == 0
    assert norm_backward(lib, M=0, dw=None) == OK
    assert norm_backward(lib, M=-1) == SHAPE
    assert norm_backward(lib, H=40000) == LIMIT
    assert norm_backward(lib, zdt=E4M3) == SHAPE
    for name in ("dy", "z", "w", "rstd", "dx", "ws"):
        assert norm_backward(lib, **{name: None}) == NULL, name
    assert norm_backward(lib, ws_bytes=need - 1) == WS
    assert norm_backward(lib, ws=ODD) == SHAPE


def test_slot_refusals(lib):
    def permute(x=A, dt=BF16, xs=None, perm=A, M=4, k=2, H=256, out=A, outs=None, rows=8):
        return lib.moe_permute(x, dt, xs, perm, M, k, H, out, outs, rows, None)

    assert permute(M=0, x=None) == OK and permute(rows=0, out=None) == OK
    assert permute(M=-1) == SHAPE and permute(rows=-1) == SHAPE and permute(k=0) == SHAPE and permute(H=0) == SHAPE
    assert permute(M=2 ** 30, k=2) == LIMIT and permute(rows=2 ** 31) == LIMIT and permute(H=2 ** 29) == LIMIT
    assert permute(dt=F32) == SHAPE and permute(dt=E4M3, H=200) == SHAPE
    assert permute(dt=E4M3, outs=A) == NULL and permute(dt=E4M3, xs=A) == NULL
    assert permute(x=None) == NULL and permute(perm=None) == NULL and permute(out=None) == NULL

    def unpermute(y=A, perm=A, w=A, M=4, k=2, H=256, out=A, rows=8):
        return lib.moe_unpermute(y, perm, w, M, k, H, out, rows, None)

    assert unpermute(M=0, y=None) == OK
    assert unpermute(M=-1) == SHAPE and unpermute(k=0) == SHAPE and unpermute(H=-4) == SHAPE and unpermute(rows=2 ** 31) == LIMIT
    assert unpermute(y=None) == NULL and unpermute(perm=None) == NULL and unpermute(out=None) == NULL

    def backward(dout=A, y=A, perm=A, w=A, M=4, k=2, H=256, dy=A, dw=A, rows=8):
        return lib.moe_unpermute_backward(dout, y, perm, w, M, k, H, dy, dw, rows, None)

    assert backward(M=0, dout=None) == OK
    assert backward(M=2 ** 31) == LIMIT and backward(k=-1) == SHAPE
    for name in ("dout", "y", "perm", "w", "dy", "dw"):
        assert backward(**{name: None}) == NULL, name


def linear(lib, **kw):
    d = _ffi.MoeLinearDesc()
    d.rows, d.E, d.N, d.K = 64, 4, 128, 256
    d.wdt, d.act, d.ydt = _ffi.MOE_W_BF16, _ffi.MOE_ACT_NONE, BF16
    d.expert_offsets = d.expert_counts = d.x = d.y = A
    d.w = _ffi.MoeWeight(A, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return lib.moe_grouped_linear(ctypes.byref(d), None)


def test_linear_refusals(lib):
    W, fp8 = _ffi.MoeWeight, _ffi.MOE_W_FP8_E4M3
    assert lib.moe_grouped_linear(None, None) == NULL
    assert linear(lib, rows=0, x=None) == OK
    assert linear(lib, rows=-1) == SHAPE and linear(lib, rows=2 ** 31) == LIMIT
    assert linear(lib, E=0) == SHAPE and linear(lib, E=1025) == LIMIT
    assert linear(lib, N=0) == SHAPE and linear(lib, N=12) == SHAPE and linear(lib, K=100) == SHAPE
    assert linear(lib, N=2 ** 15, K=2 ** 15) == LIMIT
    assert linear(lib, K=2 ** 23, N=8) == LIMIT  # 256 rows reach 2^31 bytes
    assert linear(lib, wdt=_ffi.MOE_W_BF16_TILED) == SHAPE and linear(lib, wdt=_ffi.MOE_W_MXFP4) == SHAPE
    assert linear(lib, act=4) == SHAPE and linear(lib, act=-1) == SHAPE and linear(lib, ydt=F32) == SHAPE
    assert linear(lib, expert_offsets=None) == NULL and linear(lib, expert_counts=None) == NULL
    assert linear(lib, expert_offsets=None, expert_counts=None) == NULL  # dense needs E = 1
    assert linear(lib, x=None) == NULL and linear(lib, y=None) == NULL and linear(lib, w=W(None, None)) == NULL
    assert linear(lib, act=_ffi.MOE_ACT_SWIGLU) == NULL  # no up
    assert linear(lib, up=W(A, None)) == SHAPE and linear(lib, up_bias=A) == SHAPE
    assert linear(lib, ydt=E4M3) == NULL and linear(lib, ydt=E4M3, N=136, y_scale=A) == SHAPE
    assert linear(lib, wdt=fp8, K=200) == SHAPE and linear(lib, wdt=fp8) == NULL
    assert linear(lib, wdt=fp8, w=W(A, A)) == NULL  # no x_scale
    for name in ("x", "y", "bias", "residual", "preact"):
        assert linear(lib, **{name: ODD}) == SHAPE, name
        assert name in lib.moe_last_error().decode()
    assert linear(lib, w=W(ODD, None)) == SHAPE


def test_linear_backward_refusals(lib):
    def bx(dz=A, w=A, up=None, off=A, cnt=A, rows=64, E=4, N=128, K=256, dx=A):
        return lib.moe_grouped_linear_backward_x(dz, w, up, off, cnt, rows, E, N, K, dx, None)

    assert bx(rows=0, dz=None) == OK
    assert bx(N=4) == SHAPE and bx(K=0) == SHAPE and bx(E=2000) == LIMIT and bx(rows=-1) == SHAPE
    assert bx(off=None) == NULL and bx(dz=None) == NULL and bx(w=None) == NULL and bx(dx=None) == NULL
    assert bx(dz=ODD) == SHAPE and bx(w=ODD) == SHAPE and bx(up=ODD) == SHAPE and bx(dx=ODD) == SHAPE

    size = lib.moe_grouped_linear_backward_w_workspace_bytes
    need = size(8192, 1, 128, 256, 0, 1)
    assert need > 0 and need % (128 * (256 + 1) * 4) == 0
    assert size(64, 1, 128, 256, 0, 0) == 0 and size(8192, 128, 768, 2048, 1, 0) == 0
    assert size(8192, 1, 100, 256, 0, 0) == 0 and size(-1, 1, 128, 256, 0, 0) == 0

    def bw(dz=A, x=A, gated=0, off=None, cnt=None, rows=8192, E=1, N=128, K=256, dt=BF16, dw=A, dup=None, db=A, dupb=None, ws=A,
           ws_bytes=1 << 30):
        return lib.moe_grouped_linear_backward_w(dz, x, gated, off, cnt, rows, E, N, K, dt, dw, dup, db, dupb, ws, ws_bytes, None)

    assert bw(dt=E4M3) == SHAPE and bw(N=4) == SHAPE and bw(E=4) == NULL
    assert bw(dz=None) == NULL and bw(x=None) == NULL and bw(dw=None) == NULL
    assert bw(gated=1, dupb=A) == NULL and bw(dup=A) == SHAPE and bw(dupb=A) == SHAPE
    assert bw(gated=1, dup=A) == NULL  # db without dup_b
    assert bw(dz=ODD) == SHAPE and bw(x=ODD) == SHAPE and bw(dw=ODD) == SHAPE and bw(ws=ODD) == SHAPE
    assert bw(ws=None) == NULL and bw(ws_bytes=need - 1) == WS

    def act(dy=A, pre=A, a=_ffi.MOE_ACT_SILU, off=None, cnt=None, rows=64, E=1, N=128, dz=A):
        return lib.moe_grouped_act_backward(dy, pre, a, off, cnt, rows, E, N, dz, None)

    assert act(rows=0, dy=None) == OK
    assert act(a=0) == SHAPE and act(a=4) == SHAPE and act(N=12) == SHAPE and act(E=2) == NULL
    for name in ("dy", "pre", "dz"):
        assert act(**{name: None}) == NULL and act(**{name: ODD}) == SHAPE, name


def test_binding_refusals():
    """The Python entry points refuse wrong types and shapes before any launch
    (tensors on the host are refused by the first check of all)."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    perm = torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.moe_add_rms_norm(x, w, 1e-6),
                 lambda: moe.moe_add_rms_norm(x.float(), w, 1e-6),
                 lambda: moe.moe_add_rms_norm(x[:, ::2], w, 1e-6),
                 lambda: moe.moe_add_rms_norm_backward(x, x, w, torch.ones(4)),
                 lambda: moe.moe_permute(x, perm, 2, 8),
                 lambda: moe.moe_unpermute(x, perm, 2),
                 lambda: moe.moe_unpermute_backward(x, x, perm, torch.ones(4, 2)),
                 lambda: moe.moe_grouped_linear(x, torch.zeros(8, 256, dtype=torch.bfloat16)),
                 lambda: moe.moe_grouped_linear(x, torch.zeros(8, 256, dtype=torch.bfloat16), act="relu"),
                 lambda: moe.moe_grouped_act_backward(x, x, "none"),
                 lambda: moe.moe_grouped_linear_backward_x(x, torch.zeros(256, 8, dtype=torch.bfloat16)),
                 lambda: moe.moe_grouped_linear_backward_w(x, x)):
        with pytest.raises(ValueError):
            call()
