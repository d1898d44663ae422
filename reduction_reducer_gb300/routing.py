"""Routing of tokens to experts and its gradient (``ddp_route`` and
``ddp_route_backward`` of include/ddp_reducer.h).  Only argument marshalling
happens here; the arithmetic is the library's kernels'."""

from __future__ import annotations

import struct

from . import _lib
from .reducer import DDPError, _ERRORS, _device, _stream

torch = None       # imported by the first call, not by the package; the dtypes below then too
_DTYPES = _INT = _FLOAT = _MASK = None


def _torch():
    global torch, _DTYPES, _INT, _FLOAT, _MASK
    if torch is None:
        import torch as module
        _DTYPES = {module.float32: _lib.DDP_F32, module.bfloat16: _lib.DDP_BF16}
        _INT, _FLOAT, _MASK = (module.int32,), (module.float32,), (module.bool, module.uint8)
        torch = module
    return torch


def _args(logits, k, score, groups, top_groups, renorm, scale):
    """(packed ddp_route_args, tokens, experts, the current device) of a call."""
    if torch is None:
        _torch()
    dtype, device = _DTYPES.get(logits.dtype), _device()
    if dtype is None or logits.dim() != 2 or logits.get_device() != device:
        raise ValueError(f"logits: expected [tokens, experts] fp32 or bf16 on {_found(device, logits)}")
    tokens, experts = logits.shape
    stride = _row_stride("logits", logits, tokens, experts)
    try:
        a = _lib.pack_route(tokens, stride, experts, k, _SCORES[score], groups,
                            groups if top_groups is None else top_groups, 1 if renorm else 0, scale, dtype)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"k, groups, top_groups or scale: {e}") from None
    return a, tokens, experts, device


def _row_stride(name, t, tokens, experts):
    row, column = t.stride()
    if column != 1 and experts > 1:
        raise ValueError(f"{name}: expected a token's experts next to one another")
    return row if tokens > 1 else max(row, experts)


def _found(device, t):
    return f"the current device cuda:{device}; found {list(t.shape)} of {t.dtype} on {t.device}"


def _data(name, t, shape, dtypes, device):
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name}: expected {list(shape)} contiguous {' or '.join(map(str, dtypes))} on {_found(device, t)}")
    return t.data_ptr()


class _Scores(dict):
    def __missing__(self, score):
        raise ValueError("score: expected 'softmax' or 'sigmoid'")


_SCORES = _Scores(softmax=0, sigmoid=1)


def _empty(shape, dtype, like, stream):
    """Memory of the stream that the kernel runs on: memory that was freed on
    torch's current stream may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _refused(st: int, what: str, tokens, experts, k, **more):
    detail = ", ".join(f"{n} {v}" for n, v in dict(tokens=tokens, experts=experts, k=k, **more).items())
    raise _ERRORS.get(st, DDPError)(st, f"{what}: {detail}")


def route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups=None, renorm: bool = False,
          scale: float = 1.0, mask=None, counts=None, out=None, stream=None, lib_path: str = _lib.LIB_PATH):
    """The k experts of every token and their weights: (indices int32
    [tokens, k], weights fp32 [tokens, k]).

    logits: [tokens, experts] fp32 or bf16 (rows may be strided); score:
    "softmax" or "sigmoid"; bias: fp32 [experts], added for the choice alone;
    groups, top_groups: only the top_groups best of `groups` equal runs of
    experts stay (worth: the sum of their two best); renorm: weights over
    their sum; mask: bytes or truth values [tokens], 0 = not routed (index
    -1, weight 0); counts: int32 [experts], the tokens each expert got are
    added to it; out: (indices, weights) to write into (without it they are
    allocated on `stream`).  All tensors lie on the current device."""
    a, tokens, experts, device = _args(logits, k, score, groups, top_groups, renorm, scale)
    shape, each = (tokens, k), (experts,)
    indices, weights = out if out is not None else (
        _empty(shape, torch.int32, logits, stream), _empty(shape, torch.float32, logits, stream))
    st = _lib.load(lib_path).ddp_route(
        a, logits.data_ptr(), _data("bias", bias, each, _FLOAT, device), _data("mask", mask, (tokens,), _MASK, device),
        _data("indices", indices, shape, _INT, device), _data("weights", weights, shape, _FLOAT, device),
        _data("counts", counts, each, _INT, device), _stream(stream))
    if st:
        _refused(st, "ddp_route", tokens, experts, k, groups=groups, top_groups=top_groups, scale=scale)
    return indices, weights


def route_backward(grad_weights, logits, indices, weights, score: str = "softmax", renorm: bool = False,
                   scale: float = 1.0, out=None, stream=None, lib_path: str = _lib.LIB_PATH):
    """The gradient of the logits ([tokens, experts], their dtype) from that of
    the weights, with the indices and weights that ``route`` returned for the
    same score, renorm and scale."""
    k = indices.shape[1] if indices.dim() == 2 else 0
    a, tokens, experts, device = _args(logits, k, score, 1, 1, renorm, scale)
    shape = (tokens, k)
    grad = out if out is not None else _empty((tokens, experts), logits.dtype, logits, stream)
    if grad.shape != logits.shape or grad.dtype is not logits.dtype or grad.get_device() != device:
        raise ValueError(f"out: expected the logits' shape and dtype on {_found(device, grad)}")
    st = _lib.load(lib_path).ddp_route_backward(
        a, logits.data_ptr(), _data("indices", indices, shape, _INT, device), _data("weights", weights, shape, _FLOAT, device),
        _data("grad_weights", grad_weights, shape, _FLOAT, device), grad.data_ptr(), _row_stride("out", grad, tokens, experts),
        _stream(stream))
    if st:
        _refused(st, "ddp_route_backward", tokens, experts, k, scale=scale)
    return grad


_Routed = None     # the autograd function, made on first use (torch is imported by the calls, not by the package)


def _autograd():
    global _Routed
    if _Routed is None:
        _torch()

        class Routed(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, k, options):
                indices, weights = route(logits, k, **options)
                ctx.save_for_backward(logits, indices, weights)
                ctx.options = {n: options[n] for n in ("score", "renorm", "scale", "lib_path") if n in options}
                ctx.mark_non_differentiable(indices)
                return indices, weights

            @staticmethod
            @torch.autograd.function.once_differentiable      # a second derivative raises
            def backward(ctx, _indices, grad_weights):
                logits, indices, weights = ctx.saved_tensors
                grad = route_backward(grad_weights.contiguous(), logits, indices, weights, **ctx.options)
                return grad, None, None

        _Routed = Routed
    return _Routed


def routed(logits, k: int, **options):
    """``route`` under autograd, on the current stream: (indices, weights),
    where the weights pass their gradient on to the logits.  Options: those of
    ``route`` but out and stream."""
    if "out" in options or "stream" in options:
        raise ValueError("routed: out and stream are not options here")
    return _autograd().apply(logits, k, options)
