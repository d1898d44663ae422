"""Refusals of the embedding, layer norm, dropout and log probability calls that need no GPU: every argument is checked
before anything runs."""

import ctypes as C
import os

import pytest
import torch

from reduction_reducer_gb300 import (InvalidArg, _lib, drop, dropped, embed, embed_backward, embedded, layer_norm,
                                     layer_norm_backward, layer_normed, logprobs, logprobs_backward, scored)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from reduction_reducer_gb300 import build
        build.build()
    return _lib.load()


def embed_args(**change):
    return _lib.EmbedArgs(**{**dict(tokens=4, vocab=9, dim=8, table_stride=8, row_stride=8, scale=1.0, table_dtype=0, dtype=0,
                                    index_bits=64), **change})


def norm_args(**change):
    return _lib.LayerNormArgs(**{**dict(rows=4, dim=8, x_stride=8, out_stride=8, eps=1e-5, dtype=0, param_dtype=0), **change})


def drop_args(**change):
    return _lib.DropArgs(**{**dict(rows=4, cols=8, x_stride=8, residual_stride=8, out_stride=8, p=0.5, seed=1, offset=0,
                                   device_seed=None, dtype=0), **change})


def logp_args(**change):
    return _lib.LogprobsArgs(**{**dict(rows=4, vocab=8, row_stride=8, top=2, index_bits=64, scale=1.0, dtype=0), **change})


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(tokens=2 ** 31), dict(vocab=0), dict(vocab=2 ** 31 - 1), dict(dim=0),
                                 dict(dim=2 ** 24 + 1, table_stride=2 ** 25, row_stride=2 ** 25), dict(table_stride=7),
                                 dict(row_stride=7), dict(scale=NAN), dict(scale=INF), dict(table_dtype=2), dict(dtype=-1),
                                 dict(index_bits=16)])
def test_embed_refusals(lib, bad):
    a = C.byref(embed_args(**bad))
    assert lib.ddp_embed(a, 64, 64, 64, None) == -1
    assert lib.ddp_embed_workspace(a) == -1
    assert lib.ddp_embed_backward(a, 64, 64, 64, 0, 64, None) == -1


def test_embed_pointer_refusals(lib):
    a = C.byref(embed_args())
    for call in ((None, 64, 64, 64), (a, None, 64, 64), (a, 64, None, 64), (a, 64, 64, None), (a, 66, 64, 64), (a, 64, 68, 64),
                 (a, 64, 64, 66)):
        assert lib.ddp_embed(*call, None) == -1
    for call in ((None, 64, 64, 64, 0, 64), (a, None, 64, 64, 0, 64), (a, 64, None, 64, 0, 64), (a, 64, 64, None, 0, 64),
                 (a, 64, 64, 64, 0, None), (a, 64, 64, 64, 0, 72), (a, 64, 64, 66, 0, 64), (a, 66, 64, 64, 0, 64)):
        assert lib.ddp_embed_backward(*call, None) == -1
    half = C.byref(embed_args(table_dtype=1))
    assert lib.ddp_embed_backward(half, 64, 64, 64, 1, 64, None) == -1          # sums are not kept in bf16
    assert lib.ddp_embed_workspace(a) > 0
    many = C.byref(embed_args(tokens=2 ** 24 + 1))                            # of a gradient
    assert lib.ddp_embed_backward(many, 64, 64, 64, 0, 64, None) == -1 and lib.ddp_embed_workspace(many) == -1
    none = C.byref(embed_args(tokens=0))
    assert lib.ddp_embed(none, None, None, None, None) == 0 and lib.ddp_embed_workspace(none) == 0
    assert lib.ddp_embed_backward(none, None, None, 64, 1, None, None) == 0


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(dim=0), dict(dim=2 ** 24 + 1, x_stride=2 ** 25, out_stride=2 ** 25),
                                 dict(x_stride=7), dict(out_stride=7), dict(eps=-1e-5), dict(eps=NAN), dict(eps=INF),
                                 dict(dtype=2), dict(param_dtype=3)])
def test_norm_refusals(lib, bad):
    a = C.byref(norm_args(**bad))
    assert lib.ddp_layer_norm(a, 64, 64, 64, 64, 64, None) == -1
    assert lib.ddp_layer_norm_workspace(a) == -1
    assert lib.ddp_layer_norm_backward(a, 64, 8, 64, 64, 64, 64, 64, 64, 0, 64, None) == -1


def test_norm_pointer_refusals(lib):
    a = C.byref(norm_args())
    for call in ((None, 64, 64, 64, 64, 64), (a, None, 64, 64, 64, 64), (a, 64, 64, 64, None, 64), (a, 64, 64, 64, 64, None),
                 (a, 66, 64, 64, 64, 64), (a, 64, 66, 64, 64, 64), (a, 64, 64, 66, 64, 64), (a, 64, 64, 64, 66, 64),
                 (a, 64, 64, 64, 64, 68)):
        assert lib.ddp_layer_norm(*call, None) == -1
    good = [a, 64, 8, 64, 64, 64, 64, 64, 64, 0, 64, None]
    for at, value in ((0, None), (1, None), (1, 66), (2, 7), (3, None), (4, None), (4, 68), (5, 66), (6, 66), (7, 66), (8, 66),
                      (10, None), (10, 72)):
        bad = list(good)
        bad[at] = value
        assert lib.ddp_layer_norm_backward(*bad) == -1, at
    assert lib.ddp_layer_norm_backward(a, 64, 8, 64, 64, 64, None, None, None, 0, 64, None) == -1     # nothing asked for
    half = C.byref(norm_args(param_dtype=1))
    assert lib.ddp_layer_norm_backward(half, 64, 8, 64, 64, 64, 64, 64, 64, 1, 64, None) == -1
    none = C.byref(norm_args(rows=0))
    assert lib.ddp_layer_norm(none, None, None, None, None, None, None) == 0 and lib.ddp_layer_norm_workspace(none) == 0


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=-1), dict(x_stride=7), dict(residual_stride=7), dict(out_stride=7),
                                 dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(offset=2 ** 63), dict(dtype=2),
                                 dict(device_seed=68), dict(rows=2 ** 60, cols=2 ** 60, x_stride=2 ** 60, residual_stride=2 ** 60,
                                                            out_stride=2 ** 60)])
def test_drop_refusals(lib, bad):
    assert lib.ddp_drop(C.byref(drop_args(**bad)), 64, 64, 64, None) == -1


def test_drop_pointer_refusals(lib):
    a = C.byref(drop_args())
    for call in ((None, 64, 64, 64), (a, None, 64, 64), (a, 64, 64, None), (a, 66, 64, 64), (a, 64, 66, 64), (a, 64, 64, 66)):
        assert lib.ddp_drop(*call, None) == -1
    assert lib.ddp_drop(C.byref(drop_args(rows=0)), None, None, None, None) == 0


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(vocab=0), dict(vocab=2 ** 24 + 1, row_stride=2 ** 25), dict(row_stride=7),
                                 dict(top=-1), dict(top=9), dict(top=33, vocab=64, row_stride=64), dict(scale=0.0),
                                 dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(scale=2.0 ** -65), dict(scale=2.0 ** 65), dict(dtype=2),
                                 dict(index_bits=8)])
def test_logprobs_refusals(lib, bad):
    a = C.byref(logp_args(**bad))
    assert lib.ddp_logprobs(a, 64, 64, 64, 64, 64, 64, 64, None) == -1
    if "top" not in bad:                                       # plays no part in the gradient
        assert lib.ddp_logprobs_backward(a, 64, 64, 64, 64, 64, 64, 64, bad.get("row_stride", 64), None) == -1


def test_logprobs_pointer_refusals(lib):
    a = C.byref(logp_args())
    good = [a, 64, 64, 64, 64, 64, 64, 64, None]
    for at, value in ((0, None), (1, None), (1, 66), (2, None), (2, 68), (3, None), (3, 66), (4, 66), (5, None), (5, 68), (6, None),
                      (6, 66), (7, None), (7, 66)):
        bad = list(good)
        bad[at] = value
        assert lib.ddp_logprobs(*bad) == -1, at
    good = [a, 64, 64, 64, 64, 64, 64, 64, 8, None]
    for at, value in ((0, None), (1, None), (1, 66), (2, None), (2, 68), (3, None), (3, 68), (4, None), (4, 66), (5, 66), (6, None),
                      (6, 66), (7, None), (7, 66), (8, 7)):
        bad = list(good)
        bad[at] = value
        assert lib.ddp_logprobs_backward(*bad) == -1, at
    assert lib.ddp_logprobs_backward(a, 64, 64, 64, None, None, None, 64, 8, None) == -1              # no gradient given
    none = C.byref(logp_args(rows=0))
    assert lib.ddp_logprobs(none, None, None, None, None, None, None, None, None) == 0
    assert lib.ddp_logprobs_backward(none, None, None, None, None, None, None, None, 8, None) == 0


def test_packed_arguments_have_the_structs_layout():
    for struct, pack, values in ((_lib.EmbedArgs, _lib.pack_embed, [1, 2, 3, 4, 5, 1.5, 0, 1, 64]),
                                 (_lib.LayerNormArgs, _lib.pack_layer_norm, [1, 2, 3, 4, 0.5, 1, 0]),
                                 (_lib.DropArgs, _lib.pack_drop, [1, 2, 3, 4, 5, 0.25, 2 ** 63 + 1, 7, 64, 1]),
                                 (_lib.LogprobsArgs, _lib.pack_logprobs, [1, 2, 3, 4, 32, 0.5, 1])):
        packed = pack(*values)
        assert C.sizeof(struct) == len(packed)
        a = struct.from_buffer_copy(packed)
        assert [getattr(a, n) for n, _ in struct._fields_] == values


class On:
    """A tensor as if on GPU `index`; nothing here reads or launches anything."""

    def __init__(self, tensor, index):
        self.tensor, self.index, self.is_cuda, self.device = tensor, index, True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 4096

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def calls():
    """Each call over no rows, by the names of its tensors."""
    f, i = torch.float32, torch.int64

    def z(*shape, dtype=f):
        return torch.zeros(*shape, dtype=dtype)

    return {
        "embed": (lambda t: embed(t["table"], t["tokens"], out=t["out"]), dict(table=z(9, 8), tokens=z(0, dtype=i), out=z(0, 8))),
        "embed_backward": (lambda t: embed_backward(t["grad"], t["tokens"], t["out"], accumulate=True),
                           dict(grad=z(0, 8), tokens=z(0, dtype=i), out=z(9, 8))),
        "layer_norm": (lambda t: layer_norm(t["x"], t["weight"], t["bias"], out=t["out"], stats=t["stats"]),
                       dict(x=z(0, 8), weight=z(8), bias=z(8), out=z(0, 8), stats=z(0, 2))),
        "layer_norm_backward": (lambda t: layer_norm_backward(t["grad"], t["x"], t["stats"], t["weight"], t["grad_weight"],
                                                              t["grad_bias"], out=t["out"], accumulate=True),
                                dict(grad=z(0, 8), x=z(0, 8), stats=z(0, 2), weight=z(8), grad_weight=z(8), grad_bias=z(8),
                                     out=z(0, 8))),
        "drop": (lambda t: drop(t["x"], 0.5, t["seed"], residual=t["residual"], out=t["out"]),
                 dict(x=z(0, 8), residual=z(0, 8), out=z(0, 8), seed=z(1, dtype=i))),
        "logprobs_backward": (lambda t: logprobs_backward(t["grad_logp"], t["logits"], t["targets"], t["stats"],
                                                          entropy=t["entropy"], grad_entropy=t["grad_entropy"], out=t["out"]),
                              dict(grad_logp=z(0), logits=z(0, 8), targets=z(0, dtype=i), stats=z(0, 2), entropy=z(0),
                                   grad_entropy=z(0), out=z(0, 8))),
    }


def here():
    return torch.cuda.current_device() if torch.cuda.is_available() else 0


@pytest.mark.parametrize("call,which", [(c, n) for c, (_, ts) in calls().items() for n in ts])
def test_tensors_of_another_device_are_refused(call, which):
    f, tensors = calls()[call]
    f({n: On(t, here()) for n, t in tensors.items()})
    with pytest.raises(ValueError) as e:
        f({n: On(t, here() + (n == which)) for n, t in tensors.items()})
    assert f"cuda:{here()}" in str(e.value) and f"cuda:{here() + 1}" in str(e.value)


def test_tensors_on_the_host_are_refused():
    x, t = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: embed(x, t), lambda: embedded(x, t), lambda: layer_norm(x), lambda: layer_normed(x),
                 lambda: drop(x, 0.5, 1), lambda: dropped(x, 0.5, 1), lambda: logprobs(x, t), lambda: scored(x, t)):
        with pytest.raises(ValueError, match="cpu"):
            call()


def test_shapes_types_and_layouts_are_refused():
    def on(*shape, dtype=torch.float32):
        return On(torch.zeros(*shape, dtype=dtype), here())

    i64 = torch.int64
    for call in (lambda: embed(on(9, 8), on(3, dtype=torch.int16), out=on(3, 8)),
                 lambda: embed(on(9, 8), on(3, dtype=i64), out=on(3, 9)),
                 lambda: embed(on(9, 8, dtype=torch.float16), on(3, dtype=i64), out=on(3, 8)),
                 lambda: embed(on(9, 8), on(3, dtype=i64), dtype=torch.bfloat16, out=on(3, 8)),
                 lambda: embed(on(9, 8), on(0, dtype=i64), scale="1", out=on(0, 8)),
                 lambda: embed_backward(on(4, 8), on(3, dtype=i64), on(9, 8)),
                 lambda: layer_norm(on(3, 8), on(7), out=on(3, 8), stats=on(3, 2)),
                 lambda: layer_norm(on(3, 8), on(8), on(8, dtype=torch.bfloat16), out=on(3, 8), stats=on(3, 2)),
                 lambda: layer_norm(on(3, 8), out=on(3, 8, dtype=torch.bfloat16), stats=on(3, 2)),
                 lambda: layer_norm_backward(on(3, 8), on(3, 8), on(3, 3), on(8), out=on(3, 8)),
                 lambda: drop(on(3, 8), 0.5, -1, out=on(3, 8)),
                 lambda: drop(on(3, 8), 0.5, 2 ** 64, out=on(3, 8)),
                 lambda: drop(on(3, 8), 0.5, on(2, dtype=i64), out=on(3, 8)),
                 lambda: drop(on(3, 8), 0.5, on(1), out=on(3, 8)),
                 lambda: drop(on(3, 8), 0.5, 1, residual=on(8), out=on(3, 8)),
                 lambda: logprobs_backward(on(3), on(3, 8), on(4, dtype=i64), on(3, 2), out=on(3, 8)),
                 lambda: logprobs_backward(on(3), on(3, 8), on(3, dtype=i64), on(3), out=on(3, 8)),
                 lambda: drop(On(torch.zeros(8, 3).t(), here()), 0.5, 1, out=on(3, 8)),
                 lambda: drop(On(torch.zeros(1, 8).expand(3, 8), here()), 0.5, 1, out=on(3, 8)),
                 lambda: drop(On(torch.zeros(4, 3, 16)[:, ::2, :8], here()), 0.5, 1, out=on(4, 2, 8))):
        with pytest.raises(ValueError):
            call()
    for p in (-0.5, 1.5, NAN):
        with pytest.raises(InvalidArg):
            drop(on(3, 8), p, 1, out=on(3, 8))
