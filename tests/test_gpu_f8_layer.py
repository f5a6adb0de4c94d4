"""The 8-bit operators together: the example's decode layer, eager and as a replayed graph.

Tolerance: the example's error is that of the layer from the projection's output on,
against 32 bits over the cached values: the attention (below 2^-10 of its output), its
rounding to bf16 and to e4m3 with a scale per 128 channels (relative rounding 2^-4 at
most, evenly spread: 2^-4 / sqrt(3) of the norm as an upper estimate), and y's bf16.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "f8_decode_layer.py")
BOUND = 2.0 ** -4 / 3 ** 0.5 + 2.0 ** -8 + 2.0 ** -10


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_decode_layer(window, sinks):
    spec = importlib.util.spec_from_file_location("f8_decode_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    error, us = m.run(steps=5, S=5, hidden=512, heads=2, group=4, dim=64, prompt=300, window=window, sinks=sinks)
    assert 0 < error <= BOUND
    assert us > 0
