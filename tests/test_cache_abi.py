"""gemv_qk_norm_rope, gemv_rope_frequencies and gemv_kv8_read on the host: what they
refuse, without a GPU (every call here returns before any CUDA work), and frequencies."""
from __future__ import annotations

import math

import pytest

import decode_linear_layers_gb300 as g
from tests.test_f8_abi import INVALID, UNSUPPORTED, at, built, cache  # noqa: F401  (built: a fixture)


def rope(dt=2, q=at(0), qs=1536, qo=at(1), qos=1024, qw=at(2), qh=8, k=at(0) + 2048, ks=1536, ko=at(3), kos=256, kw=at(4), kh=2, dim=128,
         eps=1e-6, freq=at(5), rot=128, layout=0, factor=1.0, lens=at(6), starts=at(7), S=3, N=6):
    return g.lib().gemv_qk_norm_rope(dt, q, qs, qo, qos, qw, qh, k, ks, ko, kos, kw, kh, dim, eps, freq, rot, layout, factor, lens,
                                     starts, S, N, None)


def read(c=None, dt=2, k=at(5), k_stride=256, v=at(6), v_stride=256, lens=at(7), starts=at(8), S=3, N=6):
    c = cache() if c is None else c
    return g.lib().gemv_kv8_read(dt, c, k, k_stride, v, v_stride, lens, starts, S, N, None)


def test_rope_refusals():
    for name in ("qh", "kh", "dim", "rot", "S", "N"):
        assert rope(**{name: -2}) == INVALID
    assert rope(dt=3) == INVALID and rope(dt=-1) == INVALID and rope(layout=2) == INVALID
    assert rope(rot=127) == INVALID and rope(rot=130) == INVALID
    assert rope(eps=-1.0) == INVALID and rope(eps=math.nan) == INVALID
    assert rope(dim=514, rot=2) == UNSUPPORTED
    assert rope(qs=1023) == INVALID and rope(ks=255) == INVALID and rope(qos=1000) == INVALID and rope(kos=0) == INVALID
    for name in ("q", "qo", "k", "ko", "freq", "lens"):
        assert rope(**{name: None}) == INVALID
    assert rope(q=at(0) + 1) == INVALID and rope(ko=at(3) + 1) == INVALID and rope(dt=0, qw=at(2) + 2) == INVALID
    assert rope(freq=at(5) + 2) == INVALID and rope(lens=at(6) + 1) == INVALID and rope(starts=at(7) + 3) == INVALID
    assert rope(starts=None, N=7) == INVALID
    assert rope(N=1 << 31) == INVALID and rope(qs=1 << 62) == INVALID
    assert rope(S=0) == 0 and rope(N=0) == 0 and rope(dim=0, rot=0) == 0 and rope(qh=0, kh=0) == 0


def test_rope_overlaps():
    # an output over an input that is not its own, in place with another stride, shifted
    assert rope(qo=at(0), qos=1024) == INVALID and rope(qo=at(0) + 256, qos=1536) == INVALID
    assert rope(ko=at(0), kos=1536) == INVALID and rope(qo=at(0) + 2048, qos=1536) == INVALID
    assert rope(ko=at(1)) == INVALID and rope(ko=at(1) + 1024, kos=1024) == INVALID
    for name in (2, 4, 5, 6, 7):
        assert rope(qo=at(name)) == INVALID and rope(ko=at(name)) == INVALID
    # columns of one matrix that share some
    assert rope(qo=at(0), qos=1536, ko=at(0) + 2046, kos=1536) == INVALID


def test_read_refusals():
    for dim in (0, 32, 96, 512):
        assert read(cache(dim=dim)) == UNSUPPORTED
    for name in ("blocks", "width", "heads", "dim"):
        assert read(cache(**{name: -1})) == INVALID
    for name in ("k", "v", "ks", "vs", "table"):
        assert read(cache(**{name: None})) == INVALID
    assert read(cache(k=at(0) + 8)) == INVALID and read(cache(ks=at(2) + 2)) == INVALID
    assert read(dt=3) == INVALID and read(S=-1) == INVALID and read(N=-1) == INVALID
    assert read(S=0) == 0 and read(N=0) == 0 and read(k=None, v=None) == 0
    assert read(starts=None, N=7) == INVALID and read(lens=None) == INVALID and read(lens=at(7) + 2) == INVALID
    assert read(k_stride=255) == INVALID and read(v_stride=0) == INVALID
    assert read(k=at(5) + 1) == INVALID and read(dt=0, v=at(6) + 2) == INVALID
    # what is written overlaps nothing; columns of one matrix that share some do
    for i in range(5):
        assert read(k=at(i)) == INVALID and read(v=at(i) + 32) == INVALID
    assert read(k=at(7)) == INVALID and read(v=at(8)) == INVALID and read(v=at(5)) == INVALID
    assert read(k_stride=600, v=at(5) + 510, v_stride=600) == INVALID and read(k_stride=600, v=at(5) + 700, v_stride=600) == INVALID


def plain(rot, base=10000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def near(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert abs(a - b) <= 2.0 ** -23 * abs(b), (a, b)


def test_frequencies():
    f, att = g.rope_frequencies(128)
    near(f, plain(128))
    assert att == 1.0
    f, att = g.rope_frequencies(64, base=5e5, scaling="linear", factor=4)
    near(f, [x / 4 for x in plain(64, 5e5)])
    assert att == 1.0
    f, _ = g.rope_frequencies(128, scaling="base", factor=8)
    assert f[0] == 1.0 and abs(f[-1] * 8 / plain(128)[-1] - 1) < 1e-6
    assert g.rope_frequencies(0) == ([], 1.0) and g.rope_frequencies(2, scaling="base", factor=3)[0] == [1.0]


def test_frequencies_by_turns():
    f, att = g.rope_frequencies(128, base=5e5, scaling="turns", factor=8, original=8192, low=1, high=4)
    want = []
    for x in plain(128, 5e5):
        wave = 2 * math.pi / x
        if wave < 8192 / 4:
            want.append(x)
        elif wave > 8192:
            want.append(x / 8)
        else:
            t = (8192 / wave - 1) / 3
            want.append((1 - t) * x / 8 + t * x)
    near(f, want)
    assert att == 1.0


def test_frequencies_by_index():
    f, att = g.rope_frequencies(128, scaling="index", factor=16, original=4096, low=1, high=32)
    pair = lambda r: 128 * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(10000))  # noqa: E731
    lo, hi = math.floor(pair(32)), math.ceil(pair(1))
    assert 0 < lo < hi < 64
    want = []
    for i, x in enumerate(plain(128)):
        ramp = min(max((i - lo) / (hi - lo), 0), 1)
        want.append(x / 16 * ramp + x * (1 - ramp))
    near(f, want)
    assert abs(att - (0.1 * math.log(16) + 1)) < 1e-6
    assert g.rope_frequencies(128, scaling="index", factor=0.5, original=4096)[1] == 1.0


def test_frequencies_refusals():
    for bad in (dict(rot=3), dict(rot=-2), dict(rot=8, base=1.0), dict(rot=8, base=math.nan), dict(rot=8, scaling="linear", factor=0),
                dict(rot=8, scaling="base", factor=math.inf), dict(rot=8, scaling="turns", factor=2),
                dict(rot=8, scaling="index", factor=2, original=100, low=4, high=4),
                dict(rot=8, scaling="index", factor=2, original=100, low=0)):
        with pytest.raises(g.GemvError) as e:
            g.rope_frequencies(**bad)
        assert e.value.status == INVALID


def prefixed(c=None, dt=2, q=at(5), q_stride=1024, lens=at(6), firsts=at(9), prefix=at(10), groups=2, out=at(7), lse=at(8), S=3, T=1,
             heads=8):
    c = cache(width=40) if c is None else c
    return g.lib().gemv_kv8_prefix_attention(dt, c, q, q_stride, lens, firsts, prefix, groups, out, lse, S, T, heads, 0.1, None)


def test_prefix_attention_refusals():
    for dim in (0, 32, 96, 512):
        assert prefixed(cache(dim=dim)) == UNSUPPORTED
    for k in ("blocks", "width", "heads", "dim"):
        assert prefixed(cache(**{k: -1})) == INVALID
    for k in ("k", "v", "ks", "vs", "table"):
        assert prefixed(cache(**{k: None})) == INVALID
    assert prefixed(cache(v=at(1) + 8)) == INVALID and prefixed(cache(vs=at(3) + 2)) == INVALID
    assert prefixed(dt=0) == INVALID and prefixed(dt=3) == INVALID
    assert prefixed(T=-1) == INVALID and prefixed(T=65) == UNSUPPORTED and prefixed(T=0) == 0
    assert prefixed(S=-1) == INVALID and prefixed(S=0) == 0
    assert prefixed(heads=7) == INVALID and prefixed(heads=-8) == INVALID and prefixed(heads=0) == 0
    assert prefixed(q_stride=1023) == INVALID
    for k in ("q", "out", "lens", "prefix"):
        assert prefixed(**{k: None}) == INVALID
    assert prefixed(groups=-1) == INVALID and prefixed(groups=4) == INVALID and prefixed(firsts=None, groups=2) == INVALID
    assert prefixed(q=at(5) + 1) == INVALID and prefixed(out=at(7) + 1) == INVALID and prefixed(lse=at(8) + 2) == INVALID
    assert prefixed(firsts=at(9) + 2) == INVALID and prefixed(prefix=at(10) + 1) == INVALID and prefixed(lens=at(6) + 2) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 9, 10):
        assert prefixed(out=at(i)) == INVALID and prefixed(lse=at(i)) == INVALID
    assert prefixed(lse=at(7)) == INVALID
