"""Argument marshalling that the operators on rows of activations share
(embedding.py, layernorm.py, dropout.py, logprobs.py)."""

from __future__ import annotations

from . import _lib
from .reducer import DDPError, _ERRORS, _device, _stream  # noqa: F401  (the operators take the latter two from here)

torch = None       # imported by the first call, not by the package; the dtypes below then too
DTYPES, CODES, INDEX = {}, {}, {}


def load_torch():
    global torch
    if torch is None:
        import torch as module
        DTYPES.update({module.float32: _lib.DDP_F32, module.bfloat16: _lib.DDP_BF16})
        CODES.update({code: dtype for dtype, code in DTYPES.items()})
        INDEX.update({module.int32: 32, module.int64: 64})
        torch = module
    return torch


def found(device, t):
    return f"the current device cuda:{device}; found {list(t.shape)} of {t.dtype} on {t.device}"


def matrix(name, t, device, shape=None, dtype=None):
    """(rows, columns, row stride, dtype's code) of a tensor of at least one
    dimension, whose last are the columns; its shape and dtype checked where
    they are given."""
    code, size = DTYPES.get(t.dtype), t.shape
    if code is None or not size or t.get_device() != device or (dtype is not None and code != dtype) or (
            shape is not None and size != shape):
        what = "fp32 or bf16" if dtype is None else str(CODES.get(dtype, "fp32 or bf16"))
        raise ValueError(f"{name}: expected {'rows' if shape is None else list(shape)} of {what} on {found(device, t)}")
    cols = size[-1]
    rows = t.numel() // cols if cols else 0
    if t.is_contiguous() or rows == 0:
        return rows, cols, cols, code
    return rows, cols, _stride(name, t, rows, cols), code


def _stride(name, t, rows, cols):
    if t.dim() != 2:
        try:
            t = t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{name}: expected rows at one distance from each other") from None
    stride, column = t.stride()
    if column != 1 and cols > 1:
        raise ValueError(f"{name}: expected a row's elements next to one another")
    if rows == 1:
        stride = cols
    if stride < cols:
        raise ValueError(f"{name}: expected rows that do not overlap")
    return stride


def vector(name, t, shape, device, dtype):
    """Address of a contiguous tensor, None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected {list(shape)} contiguous {dtype} on {found(device, t)}")
    return t.data_ptr()


def indices(name, t, shape, device, stream):
    """(tensor, address, bits) of integers.  A slice of a batch, as a next-token
    loss has them, is copied on the call's stream."""
    bits = INDEX.get(t.dtype)
    if bits is None or (shape is not None and t.shape != shape) or t.get_device() != device:
        raise ValueError(f"{name}: expected {'' if shape is None else list(shape)} int32 or int64 on {found(device, t)}")
    if not t.is_contiguous():
        with on_stream(stream):
            t = t.contiguous()
    return t, t.data_ptr(), bits


def on_stream(stream):
    """torch's current stream: the given one (None: as it is)."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def empty(shape, dtype, device, stream):
    """Memory of the stream that the kernel runs on: memory that was freed on
    torch's current stream may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def workspace(given, size, device, stream):
    """A workspace of `size` bytes: the caller's, or one of this call's."""
    if given is None:
        return empty(size, torch.uint8, device, stream)
    if given.dtype is not torch.uint8 or given.numel() < size or not given.is_contiguous() or given.get_device() != device.index:
        raise ValueError(f"workspace: expected {size} contiguous bytes on {found(device.index, given)}")
    return given


def refused(st, what, **of):
    raise _ERRORS.get(st, DDPError)(st, f"{what}: " + ", ".join(f"{n} {v}" for n, v in of.items()))


def row_gradient(t):
    """A gradient as the calls take it: what autograd hands on may be expanded."""
    if t.is_contiguous() or (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()
