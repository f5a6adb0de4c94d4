"""What the example's decode layer refuses, without a GPU (it refuses before it allocates)."""
from __future__ import annotations

import pytest

from examples import f8_decode_layer


@pytest.mark.parametrize("shared", [1, 63, 100, 8191, -64])
def test_shared_tokens_are_whole_blocks(shared):
    with pytest.raises(ValueError, match="whole number of blocks"):
        f8_decode_layer.Layer(4, 256, 2, 4, 64, 300, shared=shared)


def test_shared_tokens_have_no_window():
    with pytest.raises(ValueError, match="window"):
        f8_decode_layer.Layer(4, 256, 2, 4, 64, 300, window=100, shared=128)
