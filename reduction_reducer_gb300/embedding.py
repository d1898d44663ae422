"""Embedding of tokens and its gradient (``ddp_embed`` and
``ddp_embed_backward`` of include/ddp_reducer.h).  Only argument marshalling
happens here; the arithmetic is the library's kernels'."""

from __future__ import annotations

import struct

from . import _lib, _rows
from ._rows import _device, _stream


def _pack(n, vocab, dim, table_stride, row_stride, scale, table_code, code, bits):
    try:
        return _lib.pack_embed(n, vocab, dim, table_stride, row_stride, scale, table_code, code, bits)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"scale: {e}") from None


def embed(table, tokens, scale: float = 1.0, dtype=None, out=None, stream=None, lib_path: str = _lib.LIB_PATH):
    """scale * table[tokens]: [*tokens.shape, dim].

    table: [vocab, dim] fp32 or bf16 (rows may be strided); tokens: int32 or
    int64 of any shape (a slice is copied first); those outside [0, vocab), as
    padding is, give rows of zeros; dtype: of the result (torch.float32 or
    torch.bfloat16; the table's); out: the result's place (its rows may be
    strided).  All tensors lie on the current device."""
    if _rows.torch is None:
        _rows.load_torch()
    device = _device()
    vocab, dim, table_stride, table_code = _rows.matrix("table", table, device)
    tokens, address, bits = _rows.indices("tokens", tokens, None, device, stream)
    shape, row_stride = (*tokens.shape, dim), dim
    code = table_code if dtype is None else _rows.DTYPES.get(dtype, -1)
    if out is None and code >= 0:
        out = _rows.empty(shape, dtype or table.dtype, table.device, stream)
    else:
        _, _, row_stride, code = _rows.matrix("out", table if out is None else out, device, shape, None if dtype is None else code)
    n = tokens.numel()
    st = _lib.load(lib_path).ddp_embed(_pack(n, vocab, dim, table_stride, row_stride, scale, table_code, code, bits),
                                       table.data_ptr(), address, out.data_ptr(), _stream(stream))
    if st:
        _rows.refused(st, "ddp_embed", tokens=n, vocab=vocab, dim=dim, scale=scale)
    return out


def embed_backward(grad, tokens, out, scale: float = 1.0, accumulate: bool = False, workspace=None, stream=None,
                   lib_path: str = _lib.LIB_PATH):
    """The table's gradient, into (or, with accumulate, added to) `out`, and out.

    grad: [*tokens.shape, dim] fp32 or bf16 (rows may be strided); out:
    [vocab, dim], fp32 or, without accumulate, bf16: a gradient field or a
    bucket view (rows may be strided) that no other call writes meanwhile.  Rows without a token get zeros, and
    stay as they are with accumulate.  Sums are fp32, in the tokens' order.
    workspace: bytes that no other call uses meanwhile (without one they are
    allocated on `stream`)."""
    if _rows.torch is None:
        _rows.load_torch()
    device = _device()
    vocab, dim, table_stride, table_code = _rows.matrix("out", out, device)
    tokens, address, bits = _rows.indices("tokens", tokens, None, device, stream)
    _, _, row_stride, code = _rows.matrix("grad", grad, device, (*tokens.shape, dim))
    n, lib = tokens.numel(), _lib.load(lib_path)
    args = _pack(n, vocab, dim, table_stride, row_stride, scale, table_code, code, bits)
    size = lib.ddp_embed_workspace(args)
    st = size
    if size >= 0:
        ws = _rows.workspace(workspace, size, out.device, stream) if size else None
        st = lib.ddp_embed_backward(args, grad.data_ptr(), address, out.data_ptr(), 1 if accumulate else 0,
                                    ws.data_ptr() if size else None, _stream(stream))
    if st:
        _rows.refused(st, "ddp_embed_backward", tokens=n, vocab=vocab, dim=dim, scale=scale, accumulate=accumulate)
    return out


_Embedded = None     # the autograd function, made on first use


def _autograd():
    global _Embedded
    if _Embedded is None:
        torch = _rows.load_torch()

        class Embedded(torch.autograd.Function):
            @staticmethod
            def forward(ctx, table, tokens, scale, dtype, grad_into):
                ctx.save_for_backward(tokens)
                ctx.scale, ctx.shape, ctx.dtype, ctx.into = scale, table.shape, table.dtype, grad_into
                return embed(table, tokens, scale, dtype)

            @staticmethod
            @torch.autograd.function.once_differentiable      # a second derivative raises
            def backward(ctx, grad):
                tokens, = ctx.saved_tensors
                if ctx.into is not None:
                    embed_backward(_rows.row_gradient(grad), tokens, ctx.into, ctx.scale, accumulate=True)
                    return None, None, None, None, None
                out = torch.empty(ctx.shape, dtype=ctx.dtype, device=grad.device)
                return embed_backward(_rows.row_gradient(grad), tokens, out, ctx.scale), None, None, None, None

        _Embedded = Embedded
    return _Embedded


def embedded(table, tokens, scale: float = 1.0, dtype=None, grad_into=None):
    """``embed`` under autograd, on the current stream.  grad_into: fp32
    [vocab, dim], a gradient field or bucket view that the table's gradient is
    added to in the backward pass; autograd then gets none for the table."""
    if grad_into is not None and (grad_into.dtype is not _rows.load_torch().float32 or grad_into.shape != table.shape):
        raise ValueError(f"grad_into: expected fp32 {list(table.shape)}; found {list(grad_into.shape)} of {grad_into.dtype}")
    return _autograd().apply(table, tokens, scale, dtype, grad_into)
