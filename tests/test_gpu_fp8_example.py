"""The 8-bit layers put together: examples/fp8_layers.py."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "fp8_layers.py")
    spec = importlib.util.spec_from_file_location("fp8_layers", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_converges(ex):
    losses = ex.train(20, 384, 300)
    # each step removes about half of the error until the quantisation of x and W is left:
    # two roundings to 4 significant bits, each off by 2^-4 / sqrt(3) at most on average
    assert losses[-1] < 2 * (2 * (2.0 ** -4) ** 2 / 3), losses


def test_decoding_is_finite_and_repeatable(ex):
    import torch
    a, ia = ex.decode(3, 4)
    b, ib = ex.decode(3, 4)
    assert bool(torch.isfinite(a.float()).all()) and torch.equal(a, b) and torch.equal(ia, ib)
