"""Buffers that a product may and may not share, refused on the host before any launch."""

import ctypes

import pytest

from mixture_experts_routing_align_amd import _ffi

A, B, C = 0x10000, 0x20000, 0x30000  # non-NULL aligned addresses no call may dereference


@pytest.fixture(scope="module")
def lib():
    return _ffi.load()


def linear(lib, **kw):
    d = _ffi.MoeLinearDesc()
    d.rows, d.E, d.N, d.K = 64, 4, 128, 256
    d.wdt, d.act, d.ydt = _ffi.MOE_W_BF16, _ffi.MOE_ACT_NONE, _ffi.MOE_DT_BF16
    d.expert_offsets = d.expert_counts = d.x = d.y = A
    d.w = _ffi.MoeWeight(A, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return lib.moe_grouped_linear(ctypes.byref(d), None)


def test_8bit_rows_over_the_residual(lib):
    """8-bit rows are half as long as the residual's: one row's codes lie over another
    row's residual, which its workgroup may still have to read."""
    assert linear(lib, ydt=_ffi.MOE_DT_E4M3, y=B, y_scale=C, residual=B) == _ffi.MOE_ERR_SHAPE
    assert "residual" in lib.moe_last_error().decode()
    rows = 64 * 128  # bytes of y; the residual has twice as many
    for y, residual in ((B, B - 2 * rows + 16), (B, B + rows - 16)):  # the last, the first 16 bytes
        assert linear(lib, ydt=_ffi.MOE_DT_E4M3, y=y, y_scale=C, residual=residual) == _ffi.MOE_ERR_SHAPE
