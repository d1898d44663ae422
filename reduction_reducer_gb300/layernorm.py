"""Layer norm and its gradient (``ddp_layer_norm`` and
``ddp_layer_norm_backward`` of include/ddp_reducer.h).  Only argument
marshalling happens here; the arithmetic is the library's kernels'."""

from __future__ import annotations

import struct

from . import _lib, _rows
from ._rows import _device, _stream


def _pack(rows, dim, x_stride, out_stride, eps, code, param_code):
    try:
        return _lib.pack_layer_norm(rows, dim, x_stride, out_stride, eps, code, param_code)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"eps: {e}") from None


def _dtype(dim, device, *named):
    """The dtype of the parameter vectors, given as (name, tensor or None): that of the first."""
    for name, t in named:
        if t is not None:
            if t.dtype not in _rows.DTYPES:
                raise ValueError(f"{name}: expected [{dim}] contiguous fp32 or bf16 on {_rows.found(device, t)}")
            return t.dtype
    return _rows.torch.float32


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stats=None, stream=None,
               lib_path: str = _lib.LIB_PATH):
    """(y, stats): y = (x - mean) / sqrt(variance + eps) * weight + bias over
    the last dimension, and fp32 [*x.shape[:-1], 2], each row's mean and
    1 / sqrt(variance + eps), which the gradient takes.

    x: fp32 or bf16 (rows may be strided); weight, bias: [dim], fp32 or bf16,
    or None, both of one dtype; out, stats: the results' places, which do not
    overlap x (without them they are allocated on `stream`).  All tensors lie on the current device."""
    torch = _rows.torch or _rows.load_torch()
    device = _device()
    rows, dim, x_stride, code = _rows.matrix("x", x, device)
    kind, each = _dtype(dim, device, ("weight", weight), ("bias", bias)), (dim,)
    out_stride = dim
    if out is None:
        out = _rows.empty(x.shape, x.dtype, x.device, stream)
    else:
        out_stride = _rows.matrix("out", out, device, x.shape, code)[2]
    if stats is None:
        stats = _rows.empty((rows, 2) if x.dim() == 2 else (*x.shape[:-1], 2), torch.float32, x.device, stream)
        at = stats.data_ptr()
    else:
        at = _rows.vector("stats", stats, (*x.shape[:-1], 2), device, torch.float32)
    st = _lib.load(lib_path).ddp_layer_norm(
        _pack(rows, dim, x_stride, out_stride, eps, code, _rows.DTYPES[kind]), x.data_ptr(),
        _rows.vector("weight", weight, each, device, kind), _rows.vector("bias", bias, each, device, kind), out.data_ptr(), at,
        _stream(stream))
    if st:
        _rows.refused(st, "ddp_layer_norm", rows=rows, dim=dim, eps=eps)
    return out, stats


def layer_norm_backward(grad, x, stats, weight=None, grad_weight=None, grad_bias=None, out=None, input_grad: bool = True,
                        accumulate: bool = False, workspace=None, stream=None, lib_path: str = _lib.LIB_PATH):
    """(grad_x, grad_weight, grad_bias) from the gradient of y and the stats
    that ``layer_norm`` gave.

    grad_weight, grad_bias: [dim] of the parameters' dtype, which are written
    (or, with accumulate and fp32, added to) where they are given: gradient
    fields or bucket views; out: the place of grad_x, which overlaps neither
    grad nor x; input_grad: False
    leaves grad_x out (None); workspace: bytes that no other call uses
    meanwhile (without one they are allocated on `stream`)."""
    torch = _rows.torch or _rows.load_torch()
    device = _device()
    rows, dim, x_stride, code = _rows.matrix("x", x, device)
    _, _, grad_stride, _ = _rows.matrix("grad", grad, device, x.shape, code)
    kind, each = _dtype(dim, device, ("weight", weight), ("grad_weight", grad_weight), ("grad_bias", grad_bias)), (dim,)
    w = _rows.vector("weight", weight, each, device, kind)
    gw = _rows.vector("grad_weight", grad_weight, each, device, kind)
    gb = _rows.vector("grad_bias", grad_bias, each, device, kind)
    out_stride = dim
    if not input_grad:
        out = None
        if gw is None and gb is None:
            return None, None, None
    elif out is None:
        out = _rows.empty(x.shape, x.dtype, x.device, stream)
    else:
        out_stride = _rows.matrix("out", out, device, x.shape, code)[2]
    lib = _lib.load(lib_path)
    args = _pack(rows, dim, x_stride, out_stride, 0.0, code, _rows.DTYPES[kind])
    size = lib.ddp_layer_norm_workspace(args) if gw is not None or gb is not None else 0
    st = size
    if size >= 0:
        ws = _rows.workspace(workspace, size, x.device, stream) if size else None
        st = lib.ddp_layer_norm_backward(args, grad.data_ptr(), grad_stride, x.data_ptr(),
                                         _rows.vector("stats", stats, (*x.shape[:-1], 2), device, torch.float32), w,
                                         out.data_ptr() if input_grad else None, gw, gb, 1 if accumulate else 0,
                                         ws.data_ptr() if size else None, _stream(stream))
    if st:
        _rows.refused(st, "ddp_layer_norm_backward", rows=rows, dim=dim, accumulate=accumulate)
    return out, grad_weight, grad_bias


_Normed = None     # the autograd function, made on first use


def _autograd():
    global _Normed
    if _Normed is None:
        torch = _rows.load_torch()

        class Normed(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, bias, eps, grad_into):
                y, stats = layer_norm(x, weight, bias, eps)
                ctx.save_for_backward(x, stats, weight)
                ctx.dtypes, ctx.into = [None if t is None else t.dtype for t in (weight, bias)], grad_into
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable      # a second derivative raises
            def backward(ctx, grad):
                x, stats, weight = ctx.saved_tensors
                need_x, need_w, need_b = ctx.needs_input_grad[:3]
                field_w, field_b = ctx.into or (None, None)
                added = (need_w and field_w is not None) or (need_b and field_b is not None)

                def place(need, field, dtype):      # a call adds to both: what autograd gets then begins with zeros
                    if not need:
                        return None
                    if field is not None:
                        return field
                    return (torch.zeros if added else torch.empty)(x.shape[-1:], dtype=dtype, device=x.device)

                gw, gb = place(need_w, field_w, ctx.dtypes[0]), place(need_b, field_b, ctx.dtypes[1])
                dx, gw, gb = layer_norm_backward(_rows.row_gradient(grad), x, stats, weight, gw, gb, input_grad=need_x,
                                                 accumulate=added)
                return dx, gw if field_w is None else None, gb if field_b is None else None, None, None

        _Normed = Normed
    return _Normed


def layer_normed(x, weight=None, bias=None, eps: float = 1e-5, grad_into=None):
    """``layer_norm`` under autograd, on the current stream: y.  grad_into:
    (grad_weight, grad_bias), fp32 gradient fields or bucket views that the
    gradients of parameters in fp32 are added to in the backward pass; autograd
    then gets none for them.  Where one is None, autograd gets that gradient;
    the field of a parameter that takes no gradient stays as it is."""
    if grad_into is not None:
        _rows.load_torch()
        for t in (weight, bias, *grad_into):
            if t is not None and (t.dtype is not _rows.torch.float32 or t.shape != x.shape[-1:]):
                raise ValueError(f"grad_into: expected fp32 [{x.shape[-1]}] for parameters in fp32; found {list(t.shape)} of {t.dtype}")
    return _autograd().apply(x, weight, bias, eps, grad_into)
