"""The block-scaled example runs, learns, and stays near float32: 8-bit rounding
alone is 2^-4 of a value at most, about 2.6 % of a vector of normal values, and
a product of two such operands 3.7 %."""
import importlib.util
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block128_layers.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("block128_layers", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_then_decoding(example):
    q, s, w, losses, errors = example.train_linear()
    assert losses[0] > losses[1] > losses[2]
    assert all(0 < e < 0.05 for e in errors.values()), errors
    assert example.decode_linear(q, s, w) < 0.05


def test_experts(example):
    errors = example.experts()
    assert errors["bf16"] < 4e-3                 # the rounding of Out, 2^-9 of a value at most
    assert errors["e4m3, from a graph"] < 0.06   # three 8-bit weight matrices deep
