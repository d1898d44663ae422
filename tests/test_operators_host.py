"""Refusals of the optimizer and routing entry points that need no GPU: every
argument is checked before anything runs."""

import ctypes as C
import os

import pytest
import torch

from reduction_reducer_gb300 import AdamW, InvalidArg, NotBound, _lib, route, route_backward


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from reduction_reducer_gb300 import build
        build.build()
    return _lib.load()


def test_create_refusals(lib):
    h = C.c_void_p()
    one = (C.c_int64 * 1)(5)
    assert lib.ddp_adamw_create(one, 1, 0, 32, None) == -1
    assert lib.ddp_adamw_create(one, -1, 0, 32, C.byref(h)) == -1
    assert lib.ddp_adamw_create(None, 1, 0, 32, C.byref(h)) == -1
    assert lib.ddp_adamw_create(one, 1, 2, 32, C.byref(h)) == -1
    assert lib.ddp_adamw_create(one, 1, 0, 16, C.byref(h)) == -1
    assert b"state_bits" in lib.ddp_adamw_last_error(None)
    assert lib.ddp_adamw_create((C.c_int64 * 1)(-1), 1, 0, 32, C.byref(h)) == -1
    assert not h
    assert lib.ddp_adamw_bind(None, None, None, None, None, None, None, None, None) == -1
    assert lib.ddp_adamw_step(None, None, None) == -1
    assert lib.ddp_adamw_grad_norm(None, None, None, None) == -1
    lib.ddp_adamw_destroy(None)


@pytest.mark.parametrize("bad", [dict(t=0), dict(t=1, lr=-1.0), dict(t=1, lr=float("nan")), dict(t=1, betas=(1.0, 0.9)),
                                 dict(t=1, betas=(0.9, -0.1)), dict(t=1, eps=0.0), dict(t=1, eps=1e-60),
                                 dict(t=1, max_norm=-1.0), dict(t=1, max_norm=1.0), dict(t=1, skip_nonfinite=True),
                                 dict(t=1, lr=1e300)])
def test_step_refusals(lib, bad):
    opt = AdamW([5])
    with pytest.raises(InvalidArg):
        opt.step(stream=0, **bad)


def test_step_and_norm_before_bind(lib):
    opt = AdamW([5])
    with pytest.raises(NotBound):
        opt.step(1, stream=0)
    with pytest.raises(NotBound):
        opt.grad_norm(16, stream=0)
    with pytest.raises(InvalidArg):
        opt.grad_norm(None, stream=0)


def test_bind_refusals(lib):
    def bind(dtype="f32", bits=32, **change):
        opt = AdamW([5], dtype, bits)
        a = dict(params=[64], grads=[128], exp_avg=[192], exp_avg_sq=[256])
        a.update(change)
        with pytest.raises(InvalidArg) as e:
            opt.bind(**a)
        return str(e.value)
    assert "NULL" in bind(params=[0])
    assert "NULL" in bind(grads=[0])
    assert "aligned" in bind(grads=[130])
    assert "aligned" in bind(exp_avg=[194])
    assert "master" in bind(master=[512])                          # of fp32 parameters
    assert "master" in bind("bf16")                                # missing
    assert "scales" in bind(bits=8)
    assert "scales" in bind(exp_avg_scale=[512], exp_avg_sq_scale=[512])
    assert "weight_decay" in bind(weight_decay=-0.1)
    assert "weight_decay" in bind(weight_decay=[float("nan")])
    with pytest.raises(ValueError):
        AdamW([5]).bind([64, 64], [64], [64], [64])
    with pytest.raises(ValueError):
        AdamW([5]).bind([torch.zeros(5)], [64], [64], [64])       # not on a GPU
    with pytest.raises(ValueError):
        AdamW([5], "f16")


def _route_args(**change):
    a = dict(tokens=4, row_stride=8, experts=8, k=2, score=0, groups=1, top_groups=1, renorm=0, scale=1.0, dtype=0)
    a.update(change)
    return _lib.RouteArgs(**a)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(row_stride=7), dict(experts=0), dict(experts=513, row_stride=513),
                                 dict(k=0), dict(k=9), dict(k=33, experts=64, row_stride=64), dict(score=2), dict(groups=3),
                                 dict(groups=0), dict(groups=2, top_groups=3), dict(top_groups=0),
                                 dict(groups=4, top_groups=1, k=3), dict(scale=0.0), dict(scale=float("inf")),
                                 dict(dtype=2)])
def test_route_refusals(lib, bad):
    a = _route_args(**bad)
    assert lib.ddp_route(C.byref(a), 64, None, None, 64, 64, None, None) == -1
    assert lib.ddp_route_backward(C.byref(a), 64, 64, 64, 64, 64, 512, None) == -1


def test_route_pointer_refusals(lib):
    a = _route_args()
    r = C.byref(a)
    assert lib.ddp_route(None, 64, None, None, 64, 64, None, None) == -1
    assert lib.ddp_route(r, None, None, None, 64, 64, None, None) == -1
    assert lib.ddp_route(r, 64, None, None, None, 64, None, None) == -1
    assert lib.ddp_route(r, 66, None, None, 64, 64, None, None) == -1
    assert lib.ddp_route(r, 64, 66, None, 64, 64, None, None) == -1
    assert lib.ddp_route_backward(r, 64, 64, 64, 64, None, 8, None) == -1
    assert lib.ddp_route_backward(r, 64, 64, 64, 64, 64, 7, None) == -1
    # no tokens: nothing to do, whatever the pointers
    empty = _route_args(tokens=0)
    assert lib.ddp_route(C.byref(empty), None, None, None, None, None, None, None) == 0
    assert lib.ddp_route_backward(C.byref(empty), None, None, None, None, None, 8, None) == 0
    with pytest.raises(ValueError):
        route(torch.zeros(3, 8), 2)                                # not on a GPU
    with pytest.raises(ValueError):
        route_backward(torch.zeros(3, 2), torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))


def test_packed_arguments_have_the_structs_layout():
    a = _lib.AdamWArgs.from_buffer_copy(_lib.pack_adamw(7, 1.5, 0.25, 0.5, 2.0, 3.0, 16, 32, 2 ** 63 + 5, 1))
    assert [getattr(a, n) for n, _ in _lib.AdamWArgs._fields_] == [7, 1.5, 0.25, 0.5, 2.0, 3.0, 16, 32, 2 ** 63 + 5, 1]
    assert C.sizeof(_lib.AdamWArgs) == len(_lib.pack_adamw(7, 1, 1, 1, 1, 1, 0, 0, 0, 0))
    r = _lib.RouteArgs.from_buffer_copy(_lib.pack_route(3, 70, 64, 8, 1, 4, 2, 1, 2.5, 1))
    assert [getattr(r, n) for n, _ in _lib.RouteArgs._fields_] == [3, 70, 64, 8, 1, 4, 2, 1, 2.5, 1]
    assert C.sizeof(_lib.RouteArgs) == len(_lib.pack_route(3, 70, 64, 8, 1, 4, 2, 1, 2.5, 1))
    with pytest.raises(ValueError):
        AdamW([5]).step(1, seed=-1, stream=0)
