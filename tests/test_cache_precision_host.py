"""The inputs of tests/cache_precision.py tell formats apart: a model of the kernels' roundings
stays inside its bounds with the stated formats, and leaves them with queries, or weights,
rounded to one bf16."""
import numpy as np
import pytest

from cache_precision import Inputs, round_to

# (B, H, Hk, T, d, keys)
SHAPES = [(3, 8, 2, 2, 64, 300), (2, 8, 2, 4, 128, 300), (6, 8, 2, 2, 64, 500), (16, 8, 2, 2, 128, 600),
          (2, 8, 4, 1, 256, 200)]


def _worst(x, w, bound, **fmt):
    return (np.abs(round_to(x.result(w, **fmt), "bf16") - x.result(w)) / bound).max()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_queries(shape, seed):
    x = Inputs("queries", np.random.default_rng(seed), *shape)
    w = x.stored("fp16")
    assert np.abs(x.result(w)).max() < 1e-9
    for y, p in (("bf16x2", "bf16x2"), ("bf16x2", "bf16"), ("fp16", "bf16")):
        b = x.bound(w, y, p, "bf16", shape[4])
        assert _worst(x, w, b, y_fmt=y, p_fmt=p) <= 1.0
        assert _worst(x, w, b, y_fmt="bf16", p_fmt=p) > 1.2


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_weights(shape, seed):
    x = Inputs("weights", np.random.default_rng(seed), *shape)
    w = x.stored("fp16")
    b = x.bound(w, "bf16x2", "bf16x2", "bf16", shape[4])
    assert _worst(x, w, b, y_fmt="bf16x2", p_fmt="bf16x2") <= 1.0
    assert _worst(x, w, b, y_fmt="bf16x2", p_fmt="bf16") > 1.5


def test_rounding():
    import torch
    x = np.random.default_rng(0).standard_normal(1000) * 2.0 ** np.arange(-20, 20).repeat(25)
    assert np.array_equal(round_to(x, "bf16"), torch.from_numpy(x).bfloat16().double().numpy())
