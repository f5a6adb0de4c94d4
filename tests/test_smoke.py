"""smoke()'s own checks, without a GPU: everything that would run there is a stand-in that
counts launches as the library would."""
from __future__ import annotations

import pytest
import torch

import __graft_entry__ as entry
import decode_linear_layers_gb300 as g
import workloads as W
from examples import f8_decode_layer
from tests import gpu_util as U


@pytest.fixture
def launches(monkeypatch):
    """Launches of each GEMV and of the layer; count: those so far."""
    n = {"gemv": 1, "layer": 16, "count": 0, "gemvs": 0}

    def gemv(*a):
        n["gemvs"] += 1
        n["count"] += n["gemv"] if n["gemvs"] != n.get("none_at") else 0

    def layer(**k):
        n["count"] += n["layer"]
        return 0.01, 1.0

    for f in ("set_device", "synchronize"):
        monkeypatch.setattr(torch.cuda, f, lambda *a: None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(W, "small", lambda *a, **k: None)
    monkeypatch.setattr(W, "make_inputs", lambda *a: None)
    monkeypatch.setattr(U, "oracle_for", lambda *a: (None, None))
    monkeypatch.setattr(U, "to_device", lambda *a: None)
    monkeypatch.setattr(U, "assert_close", lambda *a, **k: None)
    monkeypatch.setattr(U, "run_gpu", gemv)
    monkeypatch.setattr(f8_decode_layer, "run", layer)
    monkeypatch.setattr(g, "launch_count", lambda: n["count"])
    return n


def test_smoke_passes_when_everything_launches(launches, capsys):
    entry.smoke()
    assert "22 libgemv kernel launches" in capsys.readouterr().out


@pytest.mark.parametrize("what", [{"gemv": 0}, {"none_at": 4}, {"layer": 0}, {"layer": 10}])
def test_smoke_fails_when_something_does_not_launch(launches, what):
    launches.update(what)
    with pytest.raises(RuntimeError, match="launch"):
        entry.smoke()
