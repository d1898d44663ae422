"""Log probabilities of given tokens with the entropy and the best
alternatives, and the gradient of their logits (``ddp_logprobs`` and
``ddp_logprobs_backward`` of include/ddp_reducer.h).  Only argument marshalling
happens here; the arithmetic is the library's kernels'."""

from __future__ import annotations

import struct
from typing import NamedTuple

from . import _lib, _rows
from ._rows import _device, _stream


class LogProbs(NamedTuple):
    """What ``logprobs`` gives; None for what was not asked for."""
    logp: object          # fp32 [...]: of the targets
    entropy: object       # fp32 [...]
    # fp32 [..., 2]: the largest logit (times scale), and the log of the sum of e^(z - largest); the largest logit
    # itself, and minus that log, where the product is past the fp32 range
    stats: object
    top_index: object     # int32 [..., top]
    top_logp: object      # fp32 [..., top]


def _pack(rows, vocab, stride, top, bits, scale, code):
    try:
        return _lib.pack_logprobs(rows, vocab, stride, top, bits, scale, code)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"top or scale: {e}") from None


def logprobs(logits, targets=None, top: int = 0, scale: float = 1.0, entropy: bool = False, stream=None,
             lib_path: str = _lib.LIB_PATH):
    """``LogProbs`` of softmax(scale * logits) over the last dimension.

    logits: [..., vocab] fp32 or bf16, rows at one distance from each other;
    targets: [...] int32 or int64 (a slice is copied first), or None; a row
    whose target lies outside [0, vocab), as padding's does, is left out (zeros,
    alternatives -1), and so are the places of a batch that have no next token,
    without a copy of the others' logits; top: 0 .. 32 alternatives, the largest
    logits in descending order, ties to the lowest index; scale: 1 /
    temperature, 2^-64 .. 2^64; entropy: whether to give it.
    All tensors lie on the current device."""
    torch = _rows.torch or _rows.load_torch()
    device = _device()
    rows, vocab, stride, code = _rows.matrix("logits", logits, device)
    lead = logits.shape[:-1]
    at, bits = None, 64
    if targets is not None:
        targets, at, bits = _rows.indices("targets", targets, lead, device, stream)
    args = _pack(rows, vocab, stride, top, bits, scale, code)
    f32, dev, empty = torch.float32, logits.device, _rows.empty
    logp = h = index = best = logp_at = h_at = index_at = best_at = None
    stats = empty((*lead, 2), f32, dev, stream)
    if targets is not None:
        logp = empty(lead, f32, dev, stream)
        logp_at = logp.data_ptr()
    if entropy:
        h = empty(lead, f32, dev, stream)
        h_at = h.data_ptr()
    if top > 0:
        index, best = empty((*lead, top), torch.int32, dev, stream), empty((*lead, top), f32, dev, stream)
        index_at, best_at = index.data_ptr(), best.data_ptr()
    st = _lib.load(lib_path).ddp_logprobs(args, logits.data_ptr(), at, logp_at, h_at, stats.data_ptr(), index_at, best_at,
                                          _stream(stream))
    if st:
        _rows.refused(st, "ddp_logprobs", rows=rows, vocab=vocab, top=top, scale=scale)
    return LogProbs(logp, h, stats, index, best)


def logprobs_backward(grad_logp, logits, targets, stats, scale: float = 1.0, entropy=None, grad_entropy=None, out=None,
                      stream=None, lib_path: str = _lib.LIB_PATH):
    """The gradient of the logits (their shape and dtype) from those of logp
    and of the entropy (fp32; either may be None, not both), with the stats and,
    for the latter, the entropy that ``logprobs`` gave for the same targets and
    scale; zeros in the rows that were left out.  out: its place (rows may be
    strided), which may be the logits' own."""
    torch = _rows.torch or _rows.load_torch()
    device = _device()
    rows, vocab, stride, code = _rows.matrix("logits", logits, device)
    lead, f32 = logits.shape[:-1], torch.float32
    at, bits = None, 64
    if targets is not None:
        targets, at, bits = _rows.indices("targets", targets, lead, device, stream)
    if grad_entropy is None:
        entropy = None
    out_stride = vocab
    if out is None:
        out = _rows.empty(logits.shape, logits.dtype, logits.device, stream)
    else:
        out_stride = _rows.matrix("out", out, device, logits.shape, code)[2]
    st = _lib.load(lib_path).ddp_logprobs_backward(
        _pack(rows, vocab, stride, 0, bits, scale, code), logits.data_ptr(), at,
        _rows.vector("stats", stats, (*lead, 2), device, f32), _rows.vector("entropy", entropy, lead, device, f32),
        _rows.vector("grad_logp", grad_logp, lead, device, f32), _rows.vector("grad_entropy", grad_entropy, lead, device, f32),
        out.data_ptr(), out_stride, _stream(stream))
    if st:
        _rows.refused(st, "ddp_logprobs_backward", rows=rows, vocab=vocab, scale=scale)
    return out


_Scored = None     # the autograd function, made on first use


def _autograd():
    global _Scored
    if _Scored is None:
        torch = _rows.load_torch()

        class Scored(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, targets, top, scale, entropy):
                got = logprobs(logits, targets, top, scale, entropy)
                ctx.save_for_backward(logits, targets, got.stats, got.entropy)
                ctx.scale = scale
                ctx.mark_non_differentiable(*(t for t in got[2:] if t is not None))
                ctx.set_materialize_grads(False)
                return tuple(got)

            @staticmethod
            @torch.autograd.function.once_differentiable      # a second derivative raises
            def backward(ctx, grad_logp, grad_entropy, *_):
                logits, targets, stats, entropy = ctx.saved_tensors
                if grad_logp is None and grad_entropy is None:
                    return None, None, None, None, None
                dense = [None if g is None else g.contiguous() for g in (grad_logp, grad_entropy)]
                grad = logprobs_backward(dense[0], logits, targets, stats, ctx.scale, entropy, dense[1])
                return grad, None, None, None, None

        _Scored = Scored
    return _Scored


def scored(logits, targets=None, top: int = 0, scale: float = 1.0, entropy: bool = False):
    """``logprobs`` under autograd, on the current stream: its logp and entropy
    pass their gradients on to the logits."""
    return LogProbs(*_autograd().apply(logits, targets, top, scale, entropy))
