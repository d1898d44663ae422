"""AdamW over every parameter in one launch, and the gradient norm it clips by
(the ``ddp_adamw_*`` calls of include/ddp_reducer.h).

The step takes the mean gradients where a reduction left them: bucket views in
the arena or the copied-back gradients.  Only argument marshalling happens
here; the arithmetic is the library's kernels'.
"""

from __future__ import annotations

import ctypes as C
import struct

from . import _lib
from .reducer import _ERRORS, DTYPES, DDPError, _device, _stream

BLOCK = 256             # elements that share one scale of an 8-bit moment (DDP_ADAMW_BLOCK)


def _addresses(name, tensors, numel, dtypes):
    """Checked addresses, on the current device, of a list of tensors (or
    addresses), as the C ABI takes them; None for None."""
    if tensors is None:
        return None
    device = _device()
    if len(tensors) != len(numel):
        raise ValueError(f"{name}: expected {len(numel)} tensors")
    out = (C.c_void_p * max(len(numel), 1))()
    for v, (t, n) in enumerate(zip(tensors, numel)):
        if isinstance(t, int):
            out[v] = t or None
        elif t is None or t.numel() != n or t.dtype not in dtypes or not t.is_contiguous() or t.get_device() != device:
            if t is not None or n:
                raise ValueError(f"{name}[{v}]: expected {n} contiguous elements of "
                                 f"{' or '.join(str(d) for d in dtypes)} on the current device cuda:{device}{_found(t)}")
        else:
            out[v] = t.data_ptr() or None
    return out


def _found(t):
    return "" if t is None else f"; found {t.numel()} of {t.dtype} on {t.device}"


class AdamW:
    """One optimizer over P tensors (``ddp_adamw``)."""

    def __init__(self, numel, param_dtype: str = "f32", state_bits: int = 32, lib_path: str = _lib.LIB_PATH):
        """numel: element counts in registration order; param_dtype: "f32", or
        "bf16" with fp32 master copies; state_bits: 32 or 8."""
        self._h = None
        self.lib = _lib.load(lib_path)
        self.numel = [int(n) for n in numel]
        self.P = len(self.numel)
        self.param_dtype, self.state_bits = param_dtype, state_bits
        if param_dtype not in DTYPES:
            raise ValueError("param_dtype: expected 'f32' or 'bf16'")
        h = C.c_void_p()
        st = self.lib.ddp_adamw_create((C.c_int64 * max(self.P, 1))(*self.numel), self.P, DTYPES[param_dtype],
                                       int(state_bits), C.byref(h))
        if st != 0:
            raise _ERRORS.get(st, DDPError)(st, self.lib.ddp_adamw_last_error(None).decode())
        self._h = h
        self._f32 = None

    def _check(self, st: int):
        if st != 0:
            raise _ERRORS.get(st, DDPError)(st, (self.lib.ddp_adamw_last_error(self._h) or b"").decode())

    # ---------------------------------------------------------------- state
    def zero_state(self, device="cuda"):
        """The state before the first step: keyword arguments of ``bind``
        (exp_avg, exp_avg_sq and, with 8 bits, their scales), views of one
        flat buffer each in which every tensor starts on a block."""
        import torch
        rows = [-(-n // BLOCK) for n in self.numel]
        start, total = [], 0
        for r in rows:
            start.append(total)
            total += r
        m_kind, v_kind = ((torch.float8_e4m3fn, torch.float8_e5m2) if self.state_bits == 8
                          else (torch.float32, torch.float32))

        def views(kind):
            flat = torch.zeros(total * BLOCK, dtype=torch.uint8 if self.state_bits == 8 else kind, device=device)
            flat = flat.view(kind)
            return [flat[o * BLOCK:o * BLOCK + n] for o, n in zip(start, self.numel)]

        state = dict(exp_avg=views(m_kind), exp_avg_sq=views(v_kind))
        if self.state_bits == 8:
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                flat = torch.zeros(total, device=device)
                state[name] = [flat[o:o + r] for o, r in zip(start, rows)]
        return state

    # ---------------------------------------------------------------- bind
    def bind(self, params, grads, exp_avg, exp_avg_sq, weight_decay=0.0, master=None, exp_avg_scale=None,
             exp_avg_sq_scale=None):
        """Lists of P tensors on the current device (or device addresses), on
        which later calls run too.  grads: fp32; params:
        param_dtype; master: fp32, with bf16 parameters; exp_avg, exp_avg_sq:
        fp32, or with 8 bits float8_e4m3fn and float8_e5m2 (or uint8) codes
        with fp32 scales of ceil(numel / 256) elements; weight_decay: a number
        for all or one per tensor.  A CUDA graph captured before this bind is
        captured anew: it holds the earlier one's table."""
        import torch
        bf16, eight = self.param_dtype == "bf16", self.state_bits == 8
        f32 = (torch.float32,)
        decay = [float(weight_decay)] * self.P if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != self.P:
            raise ValueError(f"weight_decay: expected one number or {self.P}")
        n, blocks = self.numel, [-(-n // BLOCK) for n in self.numel]
        self._check(self.lib.ddp_adamw_bind(
            self._h, _addresses("grads", grads, n, f32),
            _addresses("params", params, n, (torch.bfloat16,) if bf16 else f32),
            _addresses("master", master, n, f32),
            _addresses("exp_avg", exp_avg, n, (torch.float8_e4m3fn, torch.uint8) if eight else f32),
            _addresses("exp_avg_sq", exp_avg_sq, n, (torch.float8_e5m2, torch.uint8) if eight else f32),
            _addresses("exp_avg_scale", exp_avg_scale, blocks, f32),
            _addresses("exp_avg_sq_scale", exp_avg_sq_scale, blocks, f32), (C.c_float * max(self.P, 1))(*decay)))
        self._keep = (params, grads, exp_avg, exp_avg_sq, master, exp_avg_scale, exp_avg_sq_scale)

    def bind_grads(self, grads):
        """Bind the gradients alone: for ``grad_norm`` without a step."""
        import torch
        self._check(self.lib.ddp_adamw_bind(self._h, _addresses("grads", grads, self.numel, (torch.float32,)), None, None,
                                            None, None, None, None, None))
        self._keep = (grads,)

    # ---------------------------------------------------------------- calls
    def _used(self, used):
        if used is None or isinstance(used, int):
            return used or 0
        if used.numel() != self.P or used.element_size() != 1 or not used.is_contiguous() or used.get_device() != _device():
            raise ValueError(f"used: expected {self.P} contiguous bytes or truth values on the current device "
                             f"cuda:{_device()}{_found(used)}")
        return used.data_ptr()

    def _norm(self, norm):
        if norm is None or isinstance(norm, int):
            return norm or 0
        # a 0-d or one-element fp32 tensor; its dtype is asked for by name once
        if norm.numel() != 1 or norm.get_device() != _device() or (
                norm.dtype is not self._f32 and str(norm.dtype) != "torch.float32"):
            raise ValueError(f"norm: expected one fp32 element on the current device cuda:{_device()}{_found(norm)}")
        self._f32 = norm.dtype
        return norm.data_ptr()

    def grad_norm(self, out, used=None, stream=None):
        """out (one fp32 element on the device) = the 2-norm of the bound
        gradients, of the tensors whose ``used`` byte is not 0; returns out."""
        self._check(self.lib.ddp_adamw_grad_norm(self._h, self._used(used), self._norm(out), _stream(stream)))
        return out

    def step(self, t: int, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, norm=None, max_norm: float = 0.0,
             used=None, seed=None, skip_nonfinite: bool = False, stream=None):
        """Step number t (from 1).  norm: device fp32 the kernel clips by with
        max_norm > 0; used: device bytes [P], tensors with 0 stay as they are;
        seed: of the 8-bit moments' rounding, another one each step (None: t; one
        and the same would hold every element at a threshold of its own for ever);
        skip_nonfinite: a norm that is not finite leaves everything as it is.
        t, lr and the seed travel with the launch: a CUDA graph replays the very
        step that it captured."""
        norm, used = self._norm(norm), self._used(used)
        try:
            args = _lib.pack_adamw(t, lr, betas[0], betas[1], eps, max_norm, norm, used,
                                   max(t, 0) if seed is None else seed, 1 if skip_nonfinite else 0)
        except (struct.error, TypeError) as e:
            raise ValueError(f"t, a hyperparameter or seed: {e}") from None
        self._check(self.lib.ddp_adamw_step(self._h, args, _stream(stream)))

    def destroy(self):
        if getattr(self, "_h", None):
            self.lib.ddp_adamw_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass
