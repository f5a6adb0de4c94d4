"""gemv_f8, gemv_f8_quantize, gemv_kv8_append and gemv_kv8_attention on the host: what
they refuse, without a GPU (every call here returns before any CUDA work)."""
from __future__ import annotations

import pytest

import decode_linear_layers_gb300 as g
from decode_linear_layers_gb300.build import build

INVALID, UNSUPPORTED = g.ERR_INVALID_VALUE, g.ERR_UNSUPPORTED
P = 1 << 32   # fake addresses, far apart
STEP = 1 << 34


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def at(i):
    return P + i * STEP


def f8(A=at(0), sa=at(1), x=at(2), sx=at(3), bias=None, y=at(4), dt=2, M=64, K=64, B=2):
    return g.lib().gemv_f8(A, sa, x, sx, bias, y, dt, M, K, B, None)


def quantize(dt=2, x=at(0), q=at(1), s=at(2), K=64, B=2):
    return g.lib().gemv_f8_quantize(dt, x, q, s, K, B, None)


def test_f8_refusals():
    for k in ("M", "K", "B"):
        assert f8(**{k: -16}) == INVALID
    assert f8(K=24) == INVALID and f8(K=8) == INVALID
    assert f8(dt=3) == INVALID and f8(dt=-1) == INVALID
    for k in ("A", "sa", "x", "sx", "y"):
        assert f8(**{k: None}) == INVALID
    assert f8(A=at(0) + 8) == INVALID and f8(x=at(2) + 1) == INVALID and f8(y=at(4) + 1) == INVALID
    assert f8(sa=at(1) + 2) == INVALID and f8(sx=at(3) + 2) == INVALID and f8(bias=at(5) + 1) == INVALID
    assert f8(y=at(0) + 64) == INVALID and f8(y=at(2)) == INVALID and f8(y=at(3)) == INVALID and f8(bias=at(4), y=at(4)) == INVALID
    assert f8(M=1 << 40, K=16) == INVALID and f8(M=1 << 30, K=1 << 30, B=1 << 30) == INVALID
    assert f8(M=0) == 0 and f8(B=0) == 0


def test_quantize_refusals():
    assert quantize(K=-1) == INVALID and quantize(B=-1) == INVALID
    assert quantize(dt=3) == INVALID
    for k in ("x", "q", "s"):
        assert quantize(**{k: None}) == INVALID
    assert quantize(x=at(0) + 1) == INVALID and quantize(dt=0, x=at(0) + 2) == INVALID and quantize(s=at(2) + 2) == INVALID
    assert quantize(q=at(0)) == INVALID and quantize(s=at(0) + 4) == INVALID and quantize(s=at(1)) == INVALID
    assert quantize(K=0) == 0 and quantize(B=0) == 0


def cache(k=at(0), v=at(1), ks=at(2), vs=at(3), table=at(4), blocks=10, width=4, heads=2, dim=128):
    return g.KV8_CACHE.pack(*(p or 0 for p in (k, v, ks, vs, table)), blocks, width, heads, dim)


def append(c=None, dt=2, k=at(5), k_stride=256, v=at(6), v_stride=256, lens=at(7), starts=at(8), S=3, N=6):
    c = cache() if c is None else c
    return g.lib().gemv_kv8_append(dt, c, k, k_stride, v, v_stride, lens, starts, S, N, None)


def attention(c=None, dt=2, q=at(5), q_stride=1024, lens=at(6), out=at(7), lse=at(8), S=3, T=1, heads=8, window=0, sinks=0):
    c = cache() if c is None else c
    return g.lib().gemv_kv8_attention(dt, c, q, q_stride, lens, out, lse, S, T, heads, 0.1, window, sinks, None)


@pytest.mark.parametrize("call", [append, attention])
def test_cache_refusals(call):
    for dim in (0, 32, 96, 512):
        assert call(cache(dim=dim)) == UNSUPPORTED
    for k in ("blocks", "width", "heads", "dim"):
        assert call(cache(**{k: -1})) == INVALID
    for k in ("k", "v", "ks", "vs", "table"):
        assert call(cache(**{k: None})) == INVALID
    assert call(cache(blocks=0)) == INVALID
    assert call(cache(k=at(0) + 8)) == INVALID and call(cache(v=at(1) + 4)) == INVALID
    assert call(cache(ks=at(2) + 2)) == INVALID and call(cache(table=at(4) + 1)) == INVALID
    assert call(cache(blocks=1 << 40)) == INVALID
    assert call(S=-1) == INVALID and call(S=0) == 0
    assert call(lens=None) == INVALID and call(lens=at(6) + 2) == INVALID


def test_append_refusals():
    assert append(dt=3) == INVALID
    assert append(N=-1) == INVALID and append(N=0) == 0
    assert append(starts=None, N=7) == INVALID                        # no whole number each
    assert append(k_stride=255) == INVALID and append(v_stride=0) == INVALID
    assert append(k=None) == INVALID and append(v=None) == INVALID
    assert append(k=at(5) + 1) == INVALID and append(dt=0, v=at(6) + 2) == INVALID
    # what is written overlaps nothing
    assert append(cache(v=at(0))) == INVALID and append(cache(vs=at(2))) == INVALID
    assert append(k=at(0)) == INVALID and append(v=at(1) + 64) == INVALID and append(cache(table=at(3))) == INVALID
    assert append(cache(ks=at(1))) == INVALID and append(lens=at(2)) == INVALID and append(starts=at(3)) == INVALID


def test_attention_refusals():
    assert attention(dt=0) == INVALID and attention(dt=3) == INVALID
    assert attention(T=-1) == INVALID and attention(T=65) == UNSUPPORTED and attention(T=0) == 0
    assert attention(heads=7) == INVALID and attention(heads=-8) == INVALID and attention(heads=0) == 0
    assert attention(window=-1) == INVALID and attention(sinks=-1) == INVALID
    assert attention(q_stride=1023) == INVALID
    assert attention(q=None) == INVALID and attention(out=None) == INVALID
    assert attention(q=at(5) + 1) == INVALID and attention(out=at(7) + 1) == INVALID and attention(lse=at(8) + 2) == INVALID
    assert attention(out=at(5)) == INVALID and attention(out=at(0)) == INVALID and attention(lse=at(7)) == INVALID
    assert attention(lse=at(4)) == INVALID


def test_cache_shapes_in_the_binding():
    import torch
    k, v = torch.zeros(2, 1, 64, 128, dtype=torch.uint8), torch.zeros(2, 1, 128, 64, dtype=torch.uint8)
    s, t = torch.zeros(2, 1), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k must be"):
        g.gemv_kv8_attention("bf16", k, k, s, s, t, k, t, k, None, 1, 1, 1, 1.0)
    with pytest.raises(ValueError, match="table must be"):
        g.gemv_kv8_append("bf16", k, v, s, s, t, k, v, t, None, 2, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.gemv_kv8_append("bf16", k, v, s, s, t, k, v, t, None, 1, 1)
