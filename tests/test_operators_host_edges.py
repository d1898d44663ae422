"""Arguments of the optimizer and routing calls that are settled before anything runs (no GPU)."""

import os

import pytest
import torch

from reduction_reducer_gb300 import AdamW, InvalidArg, NotBound, _lib, route, route_backward, routed


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from reduction_reducer_gb300 import build
        build.build()


def test_a_step_without_a_seed_takes_its_number(monkeypatch):
    packed = []
    pack = _lib.pack_adamw
    monkeypatch.setattr(_lib, "pack_adamw", lambda *a: packed.append(a) or pack(*a))
    opt = AdamW([5], state_bits=8)
    for t, how, seed in ((3, {}, 3), (2 ** 40 + 1, {}, 2 ** 40 + 1), (3, dict(seed=0), 0), (3, dict(seed=9), 9)):
        with pytest.raises(NotBound):
            opt.step(t, stream=0, **how)
        assert packed[-1][8] == seed
    for t in (0, -1):
        with pytest.raises(InvalidArg):
            opt.step(t, stream=0)
    for t in (None, 1.5, "1"):
        with pytest.raises(ValueError):
            opt.step(t, stream=0)


class On:
    """A tensor as if on GPU `index`; nothing here reads or launches anything (no tokens, no bound optimizer)."""

    def __init__(self, tensor, index):
        self.tensor, self.index, self.is_cuda, self.device = tensor, index, True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 4096

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def here_and_there():
    here = torch.cuda.current_device() if torch.cuda.is_available() else 0
    return here, here + 1


def refused(call):
    here, there = here_and_there()
    with pytest.raises(ValueError) as e:
        call()
    assert f"cuda:{here}" in str(e.value) and f"cuda:{there}" in str(e.value), e.value


@pytest.mark.parametrize("which", ["logits", "bias", "mask", "counts", "indices", "weights"])
def test_routing_refuses_tensors_of_another_device(which):
    here, there = here_and_there()
    on = {n: On(t, there if n == which else here) for n, t in dict(
        logits=torch.zeros(0, 8), bias=torch.zeros(8), mask=torch.zeros(0, dtype=torch.bool),
        counts=torch.zeros(8, dtype=torch.int32), indices=torch.zeros(0, 2, dtype=torch.int32),
        weights=torch.zeros(0, 2)).items()}
    refused(lambda: route(on["logits"], 2, bias=on["bias"], mask=on["mask"], counts=on["counts"],
                          out=(on["indices"], on["weights"])))


@pytest.mark.parametrize("which", ["logits", "indices", "weights", "grad_weights", "out"])
def test_the_routing_gradient_refuses_tensors_of_another_device(which):
    here, there = here_and_there()
    on = {n: On(t, there if n == which else here) for n, t in dict(
        logits=torch.zeros(0, 8), indices=torch.zeros(0, 2, dtype=torch.int32), weights=torch.zeros(0, 2),
        grad_weights=torch.zeros(0, 2), out=torch.zeros(0, 8)).items()}
    refused(lambda: route_backward(on["grad_weights"], on["logits"], on["indices"], on["weights"], out=on["out"]))


def test_tensors_of_one_other_device_are_refused_too():
    """All on one GPU, but not the current one, on whose stream the call would run."""
    _, there = here_and_there()
    x = On(torch.zeros(0, 8), there)
    refused(lambda: route(x, 2))
    g = On(torch.zeros(0, 2), there)
    refused(lambda: route_backward(g, x, On(torch.zeros(0, 2, dtype=torch.int32), there), g))


@pytest.mark.parametrize("which", ["params", "grads", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master"])
def test_an_optimizer_refuses_tensors_of_another_device(which):
    here, there = here_and_there()
    kinds = dict(params=torch.bfloat16, grads=torch.float32, exp_avg=torch.uint8, exp_avg_sq=torch.uint8,
                 exp_avg_scale=torch.float32, exp_avg_sq_scale=torch.float32, master=torch.float32)
    opt = AdamW([5, 7], "bf16", 8)
    lists = {n: [On(torch.zeros(1 if "scale" in n else k, dtype=d), there if n == which and k == 7 else here) for k in (5, 7)]
             for n, d in kinds.items()}
    refused(lambda: opt.bind(**lists))
    if which == "grads":
        refused(lambda: opt.bind_grads(lists["grads"]))


def test_steps_and_norms_refuse_tensors_of_another_device():
    _, there = here_and_there()
    opt = AdamW([5])
    far = On(torch.zeros(1), there)
    refused(lambda: opt.step(1, norm=far, max_norm=1.0, stream=0))
    refused(lambda: opt.step(1, used=On(torch.zeros(1, dtype=torch.uint8), there), stream=0))
    refused(lambda: opt.grad_norm(far, stream=0))
    refused(lambda: opt.grad_norm(16, used=On(torch.zeros(1, dtype=torch.bool), there), stream=0))


def test_tensors_on_the_host_are_refused():
    for call in (lambda: route(torch.zeros(3, 8), 2), lambda: routed(torch.zeros(3, 8), 2),
                 lambda: AdamW([5]).bind_grads([torch.zeros(5)]), lambda: AdamW([5]).grad_norm(torch.zeros(1), stream=0)):
        with pytest.raises(ValueError, match="cpu"):
            call()


def test_a_misaligned_norm_is_refused():
    opt = AdamW([5])
    for address in (2, 4097, 4098):
        with pytest.raises(InvalidArg, match="aligned"):
            opt.grad_norm(address, stream=0)
        with pytest.raises(InvalidArg, match="aligned"):
            opt.step(1, norm=address, max_norm=1.0, stream=0)
    with pytest.raises(NotBound):
        opt.step(1, norm=4100, max_norm=1.0, stream=0)
