"""Dropout from a counter, without a stored mask (``ddp_drop`` of
include/ddp_reducer.h).  Only argument marshalling happens here; the
arithmetic is the library's kernel's."""

from __future__ import annotations

import struct

from . import _lib, _rows
from ._rows import _device, _stream


def drop(x, p: float, seed, offset: int = 0, residual=None, out=None, stream=None, lib_path: str = _lib.LIB_PATH):
    """x / (1 - p) where an element stays, 0 where it is dropped, plus the
    residual: what stays follows from (seed, offset) and each element's place
    in x's shape alone.  The gradient of x is the same call, without a
    residual, on the gradient of the result.

    x, residual: fp32 or bf16 of one shape and dtype (rows may be strided); p:
    0 .. 1, in steps of 2^-32; seed: 0 .. 2^64 - 1, or one int64 element on the
    device, which the kernel reads (a captured call draws anew at each replay
    only with this one; it has to keep its value until the backward pass);
    offset: 0 .. 2^63 - 1, another one for each call of one seed; out: the
    result's place, which may be x or residual.  All tensors lie on the
    current device."""
    if _rows.torch is None:
        _rows.load_torch()
    device = _device()
    rows, cols, x_stride, code = _rows.matrix("x", x, device)
    residual_stride, r = cols, None
    if residual is not None:
        _, _, residual_stride, _ = _rows.matrix("residual", residual, device, x.shape, code)
        r = residual.data_ptr()
    out_stride = cols
    if out is None:
        out = _rows.empty(x.shape, x.dtype, x.device, stream)
    else:
        out_stride = _rows.matrix("out", out, device, x.shape, code)[2]
    value, address = seed, 0
    if not isinstance(seed, int):
        value, address = 0, _rows.vector("seed", seed, seed.shape, device, _rows.torch.int64)
        if seed.numel() != 1:
            raise ValueError(f"seed: expected one element; found {list(seed.shape)}")
    try:
        args = _lib.pack_drop(rows, cols, x_stride, residual_stride, out_stride, p, value, offset, address, code)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"p, seed or offset: {e}") from None
    st = _lib.load(lib_path).ddp_drop(args, x.data_ptr(), r, out.data_ptr(), _stream(stream))
    if st:
        _rows.refused(st, "ddp_drop", rows=rows, cols=cols, p=p, offset=offset)
    return out


_Dropped = None     # the autograd function, made on first use


def _autograd():
    global _Dropped
    if _Dropped is None:
        torch = _rows.load_torch()

        class Dropped(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, residual, p, seed, offset):
                y = drop(x, p, seed, offset, residual)
                ctx.how = p, seed, offset
                if not isinstance(seed, int):          # that it changed is then an error of the backward pass
                    ctx.save_for_backward(seed)
                    ctx.how = p, None, offset
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable      # a second derivative raises
            def backward(ctx, grad):
                dx = None
                if ctx.needs_input_grad[0]:
                    p, seed, offset = ctx.how
                    if seed is None:
                        seed, = ctx.saved_tensors
                    dx = drop(_rows.row_gradient(grad), p, seed, offset)
                return dx, grad if ctx.needs_input_grad[1] else None, None, None, None

        _Dropped = Dropped
    return _Dropped


def dropped(x, p: float, seed, offset: int = 0, residual=None):
    """``drop`` under autograd, on the current stream; nothing is kept for the
    backward pass but a seed on the device, which raises there if torch has
    changed it meanwhile (a replayed graph is not looked at)."""
    return _autograd().apply(x, residual, p, seed, offset)
