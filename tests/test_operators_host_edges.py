"""Arguments of the optimizer and routing calls that are settled before anything runs (no GPU)."""

import os

import pytest

from reduction_reducer_gb300 import AdamW, InvalidArg, NotBound, _lib


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
