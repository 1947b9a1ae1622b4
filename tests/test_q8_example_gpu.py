"""The training example: the 8-bit block trains as the float32 one does."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gated_mlp_example(fmt):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "gated_mlp_q8.py")
    spec = importlib.util.spec_from_file_location("gated_mlp_q8", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, apart = example.train(300, 96, 200, steps=12, micro_batches=2, format=fmt,
                                  say=lambda *_: None)
    # Relative rounding error of a value, root mean square: int8 a step of 1/64 to 1/127 of the
    # block's largest magnitude (2 to 2.5 deviations above the mean of 32 normal values), over
    # sqrt(12): up to 0.012 of a typical value; e4m3 2^-4 / sqrt(12) * 1.4 = 0.025.  A gradient
    # is a sum of products of two or three such independent values.
    assert max(apart) < (0.03 if fmt == "int8" else 0.06)
    assert losses[-1][0] < 0.9 * losses[0][0]
    assert all(abs(a - b) < 0.02 * b for a, b in losses)
