"""smoke()'s check of the operators that the 8-bit layer calls, without a GPU: stand-ins that
count launches as the library would."""
from __future__ import annotations

import pytest

import __graft_entry__ as entry
import decode_linear_layers_gb300 as g
from examples import f8_decode_layer
from tests.test_smoke import launches  # noqa: F401  (a fixture)


def layer_of(monkeypatch, launches, rope, prefix):  # noqa: F811
    """The layer's calls of the two operators, with so many launches each."""
    def counting(n):
        def call(*args, **kw):
            launches["count"] += n
        return call

    def run(**kw):
        for _ in range(4):
            g.gemv_qk_norm_rope("bf16")
        for _ in range(2):
            g.gemv_kv8_prefix_attention("bf16")
        launches["count"] += 16
        return 0.01, 1.0

    calls = counting(rope), counting(prefix)
    monkeypatch.setattr(g, "gemv_qk_norm_rope", calls[0])
    monkeypatch.setattr(g, "gemv_kv8_prefix_attention", calls[1])
    monkeypatch.setattr(f8_decode_layer, "run", run)
    return calls


@pytest.mark.parametrize("rope,prefix", [(1, 3), (0, 3), (1, 2), (1, 0), (2, 3)])
def test_the_layers_operators_have_to_launch(monkeypatch, launches, rope, prefix):  # noqa: F811
    calls = layer_of(monkeypatch, launches, rope, prefix)
    if (rope, prefix) == (1, 3):
        entry.smoke()
    else:
        with pytest.raises(RuntimeError, match="libgemv launches, not"):
            entry.smoke()
    assert (g.gemv_qk_norm_rope, g.gemv_kv8_prefix_attention) == calls
