"""Operators around the expert layer (C ABI in ``include/moe_mi355x_ops.h``):
the RMS norm in front of the router, token rows laid out by expert and brought
back, the experts' products over such rows, and the gradients of all of them.

As in the rest of the binding every function marshals arguments and launches
HIP kernels on a stream (``stream=None``: the current one); there is no autograd
here, each backward pass is a call of its own.  All tensors must live on the
current device.  Outputs not given are allocated, on the stream the call runs
on; rows of an output that belong to no expert are left as they are.

8-bit rows are ``torch.float8_e4m3fn`` codes ``[rows, C]`` with float32 scales
``[rows, C / 128]``.  ``expert_offsets`` and ``expert_counts`` are those of
:class:`AlignTables`; ``None`` for both means one expert that holds every row (a
dense projection with weights ``[1, N, K]`` or ``[N, K]``).
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _ffi
from ._ffi import (
    MOE_ACT_GELU,
    MOE_ACT_NONE,
    MOE_ACT_SILU,
    MOE_ACT_SWIGLU,
    MOE_DT_BF16,
    MOE_DT_E4M3,
    MOE_DT_F32,
    MOE_W_BF16,
    MOE_W_FP8_E4M3,
    MoeLinearDesc,
    MoeWeight,
)

ACTIVATIONS = {"none": MOE_ACT_NONE, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU, "swiglu": MOE_ACT_SWIGLU}
_STREAM_TYPES = {torch.bfloat16: MOE_DT_BF16, torch.float32: MOE_DT_F32}
BLOCK = 128


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check(rc: int) -> None:
    if rc:  # not MOE_OK
        from . import MoeError

        raise MoeError(rc, _ffi.load().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The decode-width kernels take 2-5 us, so the binding keeps its own share small:
# the raw handle of the current stream and the device index are read from torch's
# C layer (0.1 us each; torch.cuda.current_stream() builds an object, 2.8 us), and
# each tensor is checked in one expression that only a refusal looks into.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _device(t, what: str) -> int:
    """Index of the GPU `t` lives on, which must be the current one."""
    if isinstance(t, torch.Tensor):
        dev = t.get_device()
        if dev >= 0 and dev == _current_device():
            return dev
        raise ValueError(what + " must be on the current GPU")
    raise ValueError(what + " must be a tensor")


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """A tensor on the device of `like` whose memory belongs to the stream the call runs on."""
    if stream is None:
        if dtype is like.dtype:
            return like.new_empty(shape)
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _matrix(t, what: str, dtypes, shape, dev: int) -> None:
    """`t` is a contiguous tensor of one of `dtypes` and of `shape` (None: any) on device `dev`."""
    if isinstance(t, torch.Tensor):
        if t.dtype in dtypes and (shape is None or t.shape == shape) and t.is_contiguous() and t.get_device() == dev:
            return
        if t.dtype in dtypes:
            if shape is not None and t.shape != shape:
                raise ValueError(f"{what} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
            raise ValueError(f"{what} must be on the current GPU")
    raise ValueError(f"{what} must be a tensor of {' or '.join(str(d) for d in dtypes)}")


def _out(t, shape, dtype, like, stream, what: str, dev: int) -> torch.Tensor:
    if t is None:
        return _new(shape, dtype, like, stream)
    _matrix(t, what, (dtype,), shape, dev)
    return t


_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_E4M3 = torch.float8_e4m3fn
_STREAM = (torch.bfloat16, torch.float32)
_ROWS = (torch.bfloat16, _E4M3)
_WEIGHTS = (torch.bfloat16, torch.uint8, _E4M3)


# -------------------------------------------------------------------- norm --

def moe_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                     fp8: bool = False, save_rstd: bool = False, out: Optional[torch.Tensor] = None,
                     out_scale: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                     rstd: Optional[torch.Tensor] = None, stream=None):
    """z = x + residual (rounded to the residual's type), y = z (mean z^2 + eps)^(-1/2) weight.

    x is bf16 [M, H] (rows may be further than H apart), residual bf16 or
    float32 [M, H] or None, weight bf16 [H].  Returns ``(y, scale, z, rstd)``: y
    bf16, or with `fp8` 8-bit rows with their scales; z (the updated stream;
    `residual_out` may be `residual` itself) or None without a residual; rstd
    float32 [M] with `save_rstd` (or given as a buffer) for the backward pass."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and x.dtype == torch.bfloat16, "x must be bf16 [M, H]")
    M, H = x.shape
    ldx = x.stride(0) if M > 1 else H
    _need((H == 1 or x.stride(1) == 1) and ldx >= H, "x must have contiguous rows that do not overlap")
    dev = _device(x, "x")
    _matrix(weight, "weight", _BF16, (H,), dev)
    rdt = MOE_DT_BF16
    if residual is not None:
        _matrix(residual, "residual", _STREAM, (M, H), dev)
        rdt = _STREAM_TYPES[residual.dtype]
        residual_out = _out(residual_out, (M, H), residual.dtype, residual, stream, "residual_out", dev)
    else:
        _need(residual_out is None, "residual_out without residual")
    _need(not fp8 or H % BLOCK == 0, "8-bit rows need H in whole blocks of 128")
    out = _out(out, (M, H), _E4M3 if fp8 else torch.bfloat16, x, stream, "out", dev)
    if fp8:
        out_scale = _out(out_scale, (M, H // BLOCK), torch.float32, x, stream, "out_scale", dev)
    else:
        _need(out_scale is None, "out_scale without fp8")
    if save_rstd or rstd is not None:
        rstd = _out(rstd, (M,), torch.float32, x, stream, "rstd", dev)
    _check(_ffi.load().moe_add_rms_norm(
        x.data_ptr(), ldx, _ptr(residual), rdt, _ptr(residual_out), weight.data_ptr(), eps, out.data_ptr(),
        MOE_DT_E4M3 if fp8 else MOE_DT_BF16, _ptr(out_scale), _ptr(rstd), M, H, _stream(stream, dev)))
    return out, out_scale, residual_out, rstd


def moe_add_rms_norm_backward(dy: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                              dz: Optional[torch.Tensor] = None, need_dweight: bool = True,
                              dx: Optional[torch.Tensor] = None, stream=None):
    """Gradients of moe_add_rms_norm from dy (bf16) and, along the residual
    stream, dz (type of z): ``(dx, dweight)``, dx (type of z) for x and the
    residual alike, dweight float32 [H] (None without `need_dweight`).  z is what
    the forward call returned (x itself where there was no residual)."""
    dev = _device(z, "z")
    _matrix(z, "z", _STREAM, None, dev)
    _need(z.dim() == 2, "z must be [M, H]")
    M, H = z.shape
    _matrix(dy, "dy", _BF16, (M, H), dev)
    _matrix(weight, "weight", _BF16, (H,), dev)
    _matrix(rstd, "rstd", _F32, (M,), dev)
    if dz is not None:
        _matrix(dz, "dz", (z.dtype,), (M, H), dev)
    dx = _out(dx, (M, H), z.dtype, z, stream, "dx", dev)
    dweight = ws = None
    nbytes = 0
    lib = _ffi.load()
    if need_dweight:
        dweight = _new((H,), torch.float32, z, stream)
        nbytes = lib.moe_add_rms_norm_backward_workspace_bytes(M, H)
        ws = _new((nbytes,), torch.uint8, z, stream) if nbytes else None
    _check(lib.moe_add_rms_norm_backward(
        dy.data_ptr(), z.data_ptr(), _STREAM_TYPES[z.dtype], weight.data_ptr(), rstd.data_ptr(), _ptr(dz),
        dx.data_ptr(), _ptr(dweight), M, H, _ptr(ws), nbytes, _stream(stream, dev)))
    return dx, dweight


# ---------------------------------------------- rows by expert, back again --

def _slots(token_to_perm, top_k: int, dev: int) -> int:
    _matrix(token_to_perm, "token_to_perm", _I32, None, dev)
    _need(top_k >= 1 and token_to_perm.numel() % top_k == 0, "token_to_perm must hold M * top_k entries")
    return token_to_perm.numel() // top_k


def moe_permute(x: torch.Tensor, token_to_perm: torch.Tensor, top_k: int, rows: int,
                scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_scale: Optional[torch.Tensor] = None, stream=None):
    """out[token_to_perm[t*top_k + k]] = x[t]: bf16 [M, H], or 8-bit rows with
    `scale`.  `rows` is the height of the sorted matrix (the length of
    ``AlignTables.sorted_token_ids``).  Returns ``(out, out_scale)`` (None for
    bf16).  The gradient is moe_unpermute without weights."""
    dev = _device(x, "x")
    M = _slots(token_to_perm, top_k, dev)
    _matrix(x, "x", _ROWS, None, dev)
    _need(x.dim() == 2 and x.shape[0] == M, "x must be [M, H]")
    _need(rows >= 0, "rows must not be negative")
    H = x.shape[1]
    fp8 = x.dtype == _E4M3
    _need(fp8 == (scale is not None), "8-bit rows come with scales, bf16 rows without")
    if fp8:
        _need(H % BLOCK == 0, "8-bit rows need H in whole blocks of 128")
        _matrix(scale, "scale", _F32, (M, H // BLOCK), dev)
        out_scale = _out(out_scale, (rows, H // BLOCK), torch.float32, x, stream, "out_scale", dev)
    else:
        _need(out_scale is None, "out_scale without 8-bit rows")
    out = _out(out, (rows, H), x.dtype, x, stream, "out", dev)
    _check(_ffi.load().moe_permute(x.data_ptr(), MOE_DT_E4M3 if fp8 else MOE_DT_BF16, _ptr(scale),
                                   token_to_perm.data_ptr(), M, top_k, H, out.data_ptr(), _ptr(out_scale), rows,
                                   _stream(stream, dev)))
    return out, out_scale


def moe_unpermute(y: torch.Tensor, token_to_perm: torch.Tensor, top_k: int,
                  topk_weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """out[t] = sum_k w[t, k] y[token_to_perm[t*top_k + k]], bf16 [M, H], slots
    without a row skipped; without weights every weight is 1 (the gradient of
    moe_permute)."""
    dev = _device(y, "y")
    M = _slots(token_to_perm, top_k, dev)
    _matrix(y, "y", _BF16, None, dev)
    _need(y.dim() == 2, "y must be [rows, H]")
    rows, H = y.shape
    if topk_weights is not None:
        _matrix(topk_weights, "topk_weights", _F32, (M, top_k), dev)
    out = _out(out, (M, H), torch.bfloat16, y, stream, "out", dev)
    _check(_ffi.load().moe_unpermute(y.data_ptr(), token_to_perm.data_ptr(), _ptr(topk_weights), M, top_k, H,
                                     out.data_ptr(), rows, _stream(stream, dev)))
    return out


def moe_unpermute_backward(dout: torch.Tensor, y: torch.Tensor, token_to_perm: torch.Tensor,
                           topk_weights: torch.Tensor, dy: Optional[torch.Tensor] = None,
                           dweights: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the weighted moe_unpermute: ``(dy, dweights)``, dy bf16
    [rows, H] (may be `y` itself), dweights float32 [M, top_k] (0 for a slot
    without a row)."""
    dev = _device(y, "y")
    _matrix(topk_weights, "topk_weights", _F32, None, dev)
    _need(topk_weights.dim() == 2, "topk_weights must be [M, top_k]")
    M, top_k = topk_weights.shape
    _matrix(token_to_perm, "token_to_perm", _I32, None, dev)
    _need(token_to_perm.numel() == M * top_k, "token_to_perm must hold M * top_k entries")
    _matrix(y, "y", _BF16, None, dev)
    _need(y.dim() == 2, "y must be [rows, H]")
    rows, H = y.shape
    _matrix(dout, "dout", _BF16, (M, H), dev)
    dy = _out(dy, (rows, H), torch.bfloat16, y, stream, "dy", dev)
    dweights = _out(dweights, (M, top_k), torch.float32, y, stream, "dweights", dev)
    _check(_ffi.load().moe_unpermute_backward(dout.data_ptr(), y.data_ptr(), token_to_perm.data_ptr(),
                                              topk_weights.data_ptr(), M, top_k, H, dy.data_ptr(),
                                              dweights.data_ptr(), rows, _stream(stream, dev)))
    return dy, dweights


# ---------------------------------------------------- the experts' products --

def _runs(expert_offsets, expert_counts, E: int, dev: int) -> None:
    if expert_offsets is None and expert_counts is None:
        _need(E == 1, "without expert_offsets there is one expert")
        return
    _need(expert_offsets is not None and expert_counts is not None, "expert_offsets and expert_counts go together")
    _matrix(expert_counts, "expert_counts", _I32, (E,), dev)
    _matrix(expert_offsets, "expert_offsets", _I32, (E + 1,), dev)


def _expert_weight(wt, what: str, dev: int):
    """(codes or bf16 [E, N, K], scales or None, E, N, K) of a weight pair or a bare bf16 tensor."""
    w, s = wt if isinstance(wt, tuple) else (wt, None)
    _matrix(w, what, _WEIGHTS, None, dev)
    if w.dim() == 3:
        E, N, K = w.shape
    else:
        _need(w.dim() == 2, what + " must be [E, N, K] or [N, K]")
        E, (N, K) = 1, w.shape
    if w.dtype == torch.bfloat16:
        _need(s is None, "bf16 weights take no scales")
    else:
        _need(N % BLOCK == 0 and K % BLOCK == 0, "8-bit weights come in whole 128x128 blocks")
        lead = () if w.dim() == 2 else (E,)
        _need(s is not None, "8-bit weights need float32 scales, one per 128x128 block")
        _matrix(s, what + " scales", _F32, lead + (N // BLOCK, K // BLOCK), dev)
    return w, s, E, N, K


def moe_grouped_linear(x: torch.Tensor, w, expert_offsets: Optional[torch.Tensor] = None,
                       expert_counts: Optional[torch.Tensor] = None, act: str = "none", up=None,
                       bias: Optional[torch.Tensor] = None, up_bias: Optional[torch.Tensor] = None,
                       residual: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
                       fp8_out: bool = False, save_preact: bool = False, out: Optional[torch.Tensor] = None,
                       out_scale: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None, stream=None):
    """y[p] = act(W[e] x[p] + bias[e]) + residual[p] for every row p of every expert e.

    `w` is a ``(w, scale)`` pair as everywhere in this package (row-major bf16, or
    e4m3fn codes with 128x128 block scales, which take 8-bit rows `x` with
    `x_scale`) or a bare bf16 tensor.  `act`: "none", "silu", "gelu" (tanh form)
    or "swiglu", silu(W x + bias) * (W_up x + up_bias) with `up`.  Returns ``(y,
    y_scale, preact)``: y bf16 [rows, N] (may be `residual` itself), or with
    `fp8_out` (or an 8-bit `out`) 8-bit rows with their scales, in buffers of their
    own; preact, with `save_preact` or given as a buffer, the bf16 pre-activations
    ([rows, 2N] for swiglu) that moe_grouped_act_backward takes."""
    _need(act in ACTIVATIONS, "act must be one of none, silu, gelu, swiglu")
    gated = act == "swiglu"
    dev = _device(x, "x")
    wt, ws, E, N, K = _expert_weight(w, "w", dev)
    _runs(expert_offsets, expert_counts, E, dev)
    fp8 = wt.dtype != torch.bfloat16
    _need(x.dim() == 2, "x must be [rows, K]")
    rows = x.shape[0]
    _matrix(x, "x", (_E4M3,) if fp8 else _BF16, (rows, K), dev)
    _need(fp8 == (x_scale is not None), "8-bit rows come with x_scale, bf16 rows without")
    if fp8:
        _matrix(x_scale, "x_scale", _F32, (rows, K // BLOCK), dev)
    _need(gated == (up is not None), "up goes with act='swiglu'")
    ut = us = None
    if gated:
        ut, us, E2, N2, K2 = _expert_weight(up, "up", dev)
        _need((E2, N2, K2) == (E, N, K) and ut.dtype == wt.dtype, "up must match w")
    else:
        _need(up_bias is None, "up_bias goes with act='swiglu'")
    if bias is not None:
        _matrix(bias, "bias", _BF16, None, dev)
        _need(bias.numel() == E * N, "bias must be [E, N]")
    if up_bias is not None:
        _matrix(up_bias, "up_bias", _BF16, None, dev)
        _need(up_bias.numel() == E * N, "up_bias must be [E, N]")
    if residual is not None:
        _matrix(residual, "residual", _BF16, (rows, N), dev)
    fp8_out = fp8_out or (out is not None and out.dtype == _E4M3)
    _need(not fp8_out or N % BLOCK == 0, "8-bit rows need N in whole blocks of 128")
    out = _out(out, (rows, N), _E4M3 if fp8_out else torch.bfloat16, x, stream, "out", dev)
    if fp8_out:
        out_scale = _out(out_scale, (rows, N // BLOCK), torch.float32, x, stream, "out_scale", dev)
    else:
        _need(out_scale is None, "out_scale without 8-bit output")
    if save_preact or preact is not None:
        preact = _out(preact, (rows, (2 if gated else 1) * N), torch.bfloat16, x, stream, "preact", dev)
    d = MoeLinearDesc(rows, E, N, K, MOE_W_FP8_E4M3 if fp8 else MOE_W_BF16, ACTIVATIONS[act],
                      MOE_DT_E4M3 if fp8_out else MOE_DT_BF16, _ptr(expert_offsets), _ptr(expert_counts),
                      x.data_ptr(), _ptr(x_scale), MoeWeight(wt.data_ptr(), _ptr(ws)), MoeWeight(_ptr(ut), _ptr(us)),
                      _ptr(bias), _ptr(up_bias), _ptr(residual), out.data_ptr(), _ptr(out_scale), _ptr(preact))
    _check(_ffi.load().moe_grouped_linear(ctypes.byref(d), _stream(stream, dev)))
    return out, out_scale, preact


def moe_grouped_act_backward(dy: torch.Tensor, preact: torch.Tensor, act: str,
                             expert_offsets: Optional[torch.Tensor] = None,
                             expert_counts: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """The gradient of the pre-activations from that of act's result: bf16, the
    shape of `preact` (which may be `dz` itself)."""
    _need(act in ("silu", "gelu", "swiglu"), "act must be silu, gelu or swiglu")
    dev = _device(dy, "dy")
    _matrix(dy, "dy", _BF16, None, dev)
    _need(dy.dim() == 2, "dy must be [rows, N]")
    rows, N = dy.shape
    wide = 2 if act == "swiglu" else 1
    _matrix(preact, "preact", _BF16, (rows, wide * N), dev)
    E = 1 if expert_counts is None else expert_counts.numel()
    _runs(expert_offsets, expert_counts, E, dev)
    dz = _out(dz, (rows, wide * N), torch.bfloat16, preact, stream, "dz", dev)
    _check(_ffi.load().moe_grouped_act_backward(dy.data_ptr(), preact.data_ptr(), ACTIVATIONS[act],
                                                _ptr(expert_offsets), _ptr(expert_counts), rows, E, N, dz.data_ptr(),
                                                _stream(stream, dev)))
    return dz


def moe_grouped_linear_backward_x(dz: torch.Tensor, w, expert_offsets: Optional[torch.Tensor] = None,
                                  expert_counts: Optional[torch.Tensor] = None, up=None,
                                  dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dx[p] = W[e]^T dz[p], plus W_up[e]^T of dz's second half with `up` (dz
    [rows, 2N]); bf16 throughout."""
    dev = _device(dz, "dz")
    wt, _, E, N, K = _expert_weight(w, "w", dev)
    _need(wt.dtype == torch.bfloat16, "gradients take bf16 weights")
    _runs(expert_offsets, expert_counts, E, dev)
    ut = None
    if up is not None:
        ut, _, E2, N2, K2 = _expert_weight(up, "up", dev)
        _need((E2, N2, K2) == (E, N, K) and ut.dtype == wt.dtype, "up must match w")
    _need(dz.dim() == 2, "dz must be [rows, N]")
    rows = dz.shape[0]
    _matrix(dz, "dz", _BF16, (rows, N if up is None else 2 * N), dev)
    dx = _out(dx, (rows, K), torch.bfloat16, dz, stream, "dx", dev)
    _check(_ffi.load().moe_grouped_linear_backward_x(dz.data_ptr(), wt.data_ptr(), _ptr(ut), _ptr(expert_offsets),
                                                     _ptr(expert_counts), rows, E, N, K, dx.data_ptr(),
                                                     _stream(stream, dev)))
    return dx


def moe_grouped_linear_backward_w(dz: torch.Tensor, x: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None,
                                  expert_counts: Optional[torch.Tensor] = None, gated: bool = False,
                                  bias: bool = False, dtype: torch.dtype = torch.bfloat16, stream=None
                                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor],
                                             Optional[torch.Tensor]]:
    """``(dw, dup, db, dup_b)``: dw[e] = sum over the expert's rows of dz^T x,
    [E, N, K] of `dtype` (bf16 or float32); with `bias` db float32 [E, N]; with
    `gated` dz is [rows, 2N] and its second half gives dup and dup_b."""
    _need(dtype in _STREAM_TYPES, "dtype must be bfloat16 or float32")
    dev = _device(x, "x")
    _matrix(dz, "dz", _BF16, None, dev)
    _matrix(x, "x", _BF16, None, dev)
    _need(dz.dim() == 2 and x.dim() == 2 and dz.shape[0] == x.shape[0], "dz and x must have the same rows")
    rows, K = x.shape
    parts = 2 if gated else 1
    _need(dz.shape[1] % parts == 0, "dz must be [rows, 2N]")
    N = dz.shape[1] // parts
    E = 1 if expert_counts is None else expert_counts.numel()
    _runs(expert_offsets, expert_counts, E, dev)
    dw = [_new((E, N, K), dtype, x, stream) for _ in range(parts)] + [None]
    db = [_new((E, N), torch.float32, x, stream) if bias else None for _ in range(parts)] + [None]
    lib = _ffi.load()
    nbytes = lib.moe_grouped_linear_backward_w_workspace_bytes(rows, E, N, K, int(gated), int(bias))
    ws = _new((nbytes,), torch.uint8, x, stream) if nbytes else None
    _check(lib.moe_grouped_linear_backward_w(
        dz.data_ptr(), x.data_ptr(), int(gated), _ptr(expert_offsets), _ptr(expert_counts), rows, E, N, K,
        _STREAM_TYPES[dtype], dw[0].data_ptr(), _ptr(dw[1]), _ptr(db[0]), _ptr(db[1]), _ptr(ws), nbytes,
        _stream(stream, dev)))
    return dw[0], dw[1], db[0], db[1]
