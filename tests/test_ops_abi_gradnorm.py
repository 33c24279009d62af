"""Host-side refusals of gradient clipping whose norm or workspace lies over the gradients:
a launch would read what another workgroup of it writes (no compute call runs here)."""

import ctypes

import pytest

from mixture_experts_routing_align_amd import _ffi
from test_ops_abi_mxfp4 import tensors

A, B, FREE = 0x10000, 0x20000, 0x90000  # addresses no call may dereference
SHAPE, BF16, F32 = _ffi.MOE_ERR_SHAPE, _ffi.MOE_DT_BF16, _ffi.MOE_DT_F32
N = 64  # elements of each tensor


@pytest.fixture(scope="module")
def lib():
    return _ffi.load()


def refused(lib, status, what):
    return status == SHAPE and what in lib.moe_last_error().decode()


@pytest.mark.parametrize("at", [A, A + 2 * N - 4, B, B + 4 * N - 4])
def test_norm_over_a_tensor(lib, at):
    for to in ((A, B), (A + 0x4000, B + 0x4000)):  # in place, and with outputs of their own
        t = tensors((A, to[0], N, BF16), (B, to[1], N, F32))
        assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 2, 1.0, at, FREE, 1 << 20, None), "norm")
    t = tensors((A + 0x4000, A, N, BF16), (B + 0x4000, B, N, F32))  # outputs there
    assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 2, 1.0, at, FREE, 1 << 20, None), "norm")
    assert refused(lib, lib.moe_grad_clip(ctypes.addressof(t), 2, at, 1.0, None), "norm")


def test_norm_half_over_a_tensor(lib):
    for at in (A, A + 4):  # two bytes of the norm on one bf16 element
        t = tensors((A + 2, A + 2, 2, BF16))
        assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 1, 1.0, at, FREE, 1 << 20, None), "norm")


def test_workspace_over_a_tensor(lib):
    size = lib.moe_grad_norm_workspace_bytes(2)
    for ws in (A, A - size + 8, A + 2 * N - 8, B + 4 * N - 8):
        t = tensors((A, A, N, BF16), (B, B, N, F32))
        assert refused(lib, lib.moe_grad_norm(ctypes.addressof(t), 2, FREE, ws, size, None), "workspace")
        assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 2, 1.0, FREE, ws, size, None), "workspace")
        t = tensors((A + 0x4000, A, N, BF16), (B + 0x4000, B, N, F32))
        assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 2, 1.0, FREE, ws, size, None), "workspace")


def test_norm_in_the_workspace(lib):
    size = lib.moe_grad_norm_workspace_bytes(1)
    t = tensors((A, A, N, BF16))
    for norm in (FREE, FREE + size - 4):
        assert refused(lib, lib.moe_grad_norm(ctypes.addressof(t), 1, norm, FREE, size, None), "workspace")
        assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 1, 1.0, norm, FREE, size, None), "workspace")


def test_norm_alignment(lib):
    t = tensors((A, A, N, BF16))
    size = lib.moe_grad_norm_workspace_bytes(1)
    assert refused(lib, lib.moe_grad_norm(ctypes.addressof(t), 1, B + 2, FREE, size, None), "norm")
    assert refused(lib, lib.moe_grad_clip(ctypes.addressof(t), 1, B + 2, 1.0, None), "norm")
    assert refused(lib, lib.moe_clip_grad_norm(ctypes.addressof(t), 1, 1.0, B + 2, FREE, size, None), "norm")
