"""The gated MLP example: it trains, and serves its weights in 8 bits."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("size", [[], ["--tokens", "301", "--width", "264", "--hidden", "520", "--steps", "40"]])
def test_gated_mlp(size):
    pytest.importorskip("torch")
    spec = importlib.util.spec_from_file_location("gated_mlp", os.path.join(ROOT, "examples", "gated_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, error, same = m.main(size)
    # two random networks start a loss of about twice the output's variance apart
    assert losses[-1] < 0.7 * losses[0], losses
    # three roundings to 8 bits (two activations, the weights) of about 1 / 254 of a row's largest value,
    # three to four times its size: below 4 * sqrt(4) / 254 in all
    assert error < 0.04
    assert same, "rows of an 8-bit product do not depend on the batch"
