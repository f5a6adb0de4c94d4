"""The operators around the 8-bit cache together, as a served batch uses them: queries and
keys turned, keys and values appended, attention behind a shared prefix, tokens read back;
eager and as a replayed graph.

Tolerances: those of the operators' own tests, each from what the one before it really
gave (the turned queries, the cached values), so that nothing adds up; the decode layer's
as in tests/test_gpu_f8_layer.py.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g
from tests.test_gpu_f8_layer import BOUND, PATH
from tests.test_gpu_kv8 import BLOCK, E4M3, ROUND, attention_reference, gen
from tests.test_gpu_kv8_read import reference as read_reference, same
from tests.test_gpu_prefix import Shared, small_weights
from tests.test_gpu_rope import close, frequencies, reference as turned

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("name,dim,T", [("bf16", 128, 1), ("f16", 64, 3), ("bf16", 256, 2)])
def test_steps_of_a_batch(name, dim, T):
    dt = torch.bfloat16 if name == "bf16" else torch.float16
    heads, group, P = 2, 4, 448
    firsts, prefix = [0, 5, 9], [P, 320]
    lens = [P + 40, P + T, P + 63, 0, P + 1 + T, 320 + T, 400, 330, 321 + T]
    S, Hq = len(lens), heads * group
    steps = 4
    # room for the steps' tokens: the tables are those of longer sequences
    c = Shared(firsts, prefix, [n + (steps + 1) * T if n else 0 for n in lens], heads, dim, seed=dim).fill(1)
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    live = [s for s in range(S) if lens[s]]
    # the idle place has no rows: its T are another sequence's in `starts`
    counts = [T if n else 0 for n in lens]
    st = [0]
    for n in counts:
        st.append(st[-1] + n)
    starts, N = torch.tensor(st, dtype=torch.int32, device="cuda"), st[-1]
    qkv = torch.empty(N, (Hq + 2 * heads) * dim, dtype=dt, device="cuda")
    q, k, v = (x.unflatten(1, (-1, dim)) for x in (qkv[:, :Hq * dim], qkv[:, Hq * dim:(Hq + heads) * dim], qkv[:, (Hq + heads) * dim:]))
    qw, kw = ((1 + 0.2 * torch.randn(2, dim, generator=gen(2), device="cuda")).to(dt))
    freq, _ = frequencies(dim, scaling="index", factor=4, original=4096)
    rows = torch.zeros(S, T, Hq, dim, dtype=dt, device="cuda")   # queries where the attention looks for them
    where = torch.tensor([s * T + t for s in live for t in range(T)], device="cuda")
    out, lse = torch.empty_like(rows), torch.empty(S, T, Hq, device="cuda")
    back_k, back_v = torch.empty(N, heads, dim, dtype=dt, device="cuda"), torch.empty(N, heads, dim, dtype=dt, device="cuda")

    def step():
        c.lens.add_(starts[1:] - starts[:-1])
        g.gemv_qk_norm_rope(name, q, k, None, None, qw, kw, freq, c.lens, starts, S, N, Hq, heads, dim, dim, factor=1.1)
        g.gemv_kv8_append(name, *c.args(), k, v, c.lens, starts, S, N)
        rows.view(S * T, Hq, dim).index_copy_(0, where, q)
        g.gemv_kv8_prefix_attention(name, *c.args(), rows, c.lens, c.firsts, c.prefix, out, lse, S, T, Hq, 1 / math.sqrt(dim))
        g.gemv_kv8_read(name, *c.args(), back_k, back_v, c.lens, starts, S, N)

    graph = None
    for i in range(steps):
        fresh = (torch.randn(N, qkv.shape[1], generator=gen(10 + i), device="cuda") * 2).to(dt)
        qkv.copy_(fresh)
        if i == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        now = [n + (i + 1) * m for n, m in zip(lens, counts)]
        assert c.lens.tolist() == now
        pos = torch.tensor([now[s] - T + t for s in live for t in range(T)], dtype=torch.float64, device="cuda")
        fq, fk = (x.unflatten(1, (-1, dim)) for x in (fresh[:, :Hq * dim], fresh[:, Hq * dim:(Hq + heads) * dim]))
        close(name, q, *turned(fq, qw, pos, freq, dim, "half", 1e-6, 1.1))
        close(name, k, *turned(fk, kw, pos, freq, dim, "half", 1e-6, 1.1))
        want_k, want_v = read_reference(c, counts, dt, back_k, back_v)
        assert same(back_k, want_k) and same(back_v, want_v)
        # the tokens of this step, as appended: half a step of e4m3, at a scale of their block's (tests/test_gpu_kv8_read.py)
        scale = max(float(c.ks.max()), float(c.vs.max()))
        for a, b in ((k, back_k), (v, back_v)):
            err = (a.float() - b.float()).abs()
            assert bool((err <= a.float().abs() * (2.0 ** -4 + 2.0 ** -8) + 2.0 ** -10 * scale).all())
        ref, ref_lse, tol = attention_reference(c, rows, 1 / math.sqrt(dim), 0, 0)
        tol = tol + small_weights(c, rows, 1 / math.sqrt(dim))
        fine = ~torch.isnan(ref)
        assert torch.equal(~torch.isnan(out), fine)
        assert bool(((out.double() - ref).abs()[fine] <= (tol + ROUND[name] * ref.abs() + 2.0 ** -24)[fine]).all())
        assert torch.equal(lse == -math.inf, ref_lse == -math.inf) and bool((out[3] == 0).all())


@pytest.mark.parametrize("rotate,shared,prompt", [(True, 0, 300), (True, 256, 300), (False, 8192, 100)])
def test_decode_layer_with_positions_and_a_shared_prompt(rotate, shared, prompt):
    import importlib.util
    spec = importlib.util.spec_from_file_location("f8_decode_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    S, heads = (40, 4) if shared > 1000 else (5, 2)     # (the larger one is shared, the others are passed on)
    n = g.launch_count()
    error, us = m.run(steps=4, S=S, hidden=512, heads=heads, group=4, dim=128 if shared > 1000 else 64, prompt=prompt, rotate=rotate, shared=shared)
    assert 0 < error <= BOUND and us > 0
    assert g.launch_count() - n >= 12


@pytest.mark.parametrize("rotate,shared,prompt", [(True, 0, 300), (True, 256, 300), (False, 8192, 100), (True, 8192, 100)])
def test_decode_layer_launches_what_it_is_asked_for(monkeypatch, rotate, shared, prompt):
    from examples import f8_decode_layer as m
    wide = shared > 1000
    launched = {}

    def counted(name):
        call = getattr(g, name)

        def run(*a, **k):
            n = g.launch_count()
            call(*a, **k)
            launched.setdefault(name, []).append(g.launch_count() - n)
        return run

    for name in ("gemv_qk_norm_rope", "gemv_kv8_attention", "gemv_kv8_prefix_attention"):
        monkeypatch.setattr(m.g, name, counted(name))
    m.run(steps=4, S=40 if wide else 5, hidden=512, heads=4 if wide else 2, group=4, dim=128 if wide else 64, prompt=prompt, rotate=rotate,
          shared=shared)
    # the shared tokens, the prompts, an eager step and a captured one; tables of five blocks or more
    # take two kernels, the shared form three
    assert launched.pop("gemv_qk_norm_rope", []) == [1] * ((3 + (shared > 0)) if rotate else 0)
    assert launched == ({"gemv_kv8_prefix_attention": [3 if wide else 2] * 2} if shared else {"gemv_kv8_attention": [2] * 2})
