"""gemv_qk_norm_rope against the definition in 64 bits.

Tolerance.  The sum of squares is fp32, 16 terms to a lane and five steps between lanes,
all positive: 22 roundings, half of that after the root; rsqrt two units, the division and
the two products three more: below 2^-19 relative in all.  cos and sin: the angle is good
to 2^-23, the function to two units, 2^-22, and the factor's rounding 2^-24: below 2^-21.
Two products and a sum add 2^-22.  So an output y of the pair (a, b) is off by at most
(|n_a| + |n_b|) |factor| (2^-19 + 2^-21 + 2^-22), and by its own rounding.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
REL = 2.0 ** -19 + 2.0 ** -21 + 2.0 ** -22


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def positions(lens, counts):
    return torch.tensor([n - c + i for n, c in zip(lens, counts) for i in range(c)], dtype=torch.float64, device="cuda")


def reference(x, w, pos, freq, rot, layout, eps, factor):
    """(y, |n_a| + |n_b| for the bound) of rows x heads x dim, in 64 bits."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.double()
    mag = y.abs()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
    t = pos[:, None, None] * freq.double()
    na, nb = y[..., a], y[..., b]
    y, m = y.clone(), mag.clone()
    y[..., a] = factor * (na * t.cos() - nb * t.sin())
    y[..., b] = factor * (nb * t.cos() + na * t.sin())
    m[..., a] = m[..., b] = abs(factor) * (na.abs() + nb.abs())
    return y, m


def close(name, got, want, mag):
    err = (got.double() - want).abs()
    bound = REL * mag + ROUND[name] * want.abs() + (2.0 ** -25 if name == "f16" else 1e-40)
    assert bool((err <= bound).all()), float((err / bound).max())


def frequencies(rot, **kw):
    f, factor = g.rope_frequencies(rot, **kw)
    return torch.tensor(f, dtype=torch.float32, device="cuda"), factor


def check(name, lens, counts, q_heads, k_heads, dim, rot, layout, norm=True, seed=1, even=False, factor=1.25, eps=1e-5, place=False,
          gap=3):
    dt, N, S = TYPES[name], sum(counts), len(lens)
    width = (q_heads + 2 * k_heads) * dim + gap
    qkv = (torch.randn(N, width, generator=gen(seed), device="cuda") * 3).to(dt)
    q, k = qkv[:, :q_heads * dim].unflatten(1, (q_heads, dim)), qkv[:, q_heads * dim:(q_heads + k_heads) * dim].unflatten(1, (k_heads, dim))
    qw, kw = ((1 + torch.randn(dim, generator=gen(seed + 1 + j), device="cuda")).to(dt) if norm else None for j in range(2))
    freq, _ = frequencies(rot)
    pos = positions(lens, counts)
    want = [reference(x, w, pos, freq, rot, layout, eps, factor) for x, w in ((q, qw), (k, kw))]
    before = qkv.clone()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = None if even else offsets(counts)
    out = torch.full_like(qkv, 7.0)
    qo, ko = (None, None) if place else (out[:, :q_heads * dim].unflatten(1, (q_heads, dim)),
                                         out[:, q_heads * dim:(q_heads + k_heads) * dim].unflatten(1, (k_heads, dim)))
    call = lambda: g.gemv_qk_norm_rope(name, q, k, qo, ko, qw, kw, freq if rot else None, lens_t, starts, S, N, q_heads, k_heads,  # noqa: E731
                                       dim, rot, layout=layout, eps=eps, factor=factor)
    call()
    torch.cuda.synchronize()
    if place:
        qo, ko = q, k
        assert torch.equal(qkv[:, (q_heads + k_heads) * dim:], before[:, (q_heads + k_heads) * dim:])
    else:
        assert torch.equal(qkv, before) and bool((out[:, (q_heads + k_heads) * dim:] == 7).all())
    for got, (y, m) in zip((qo, ko), want):
        close(name, got, y, m)
    if not place:
        first = out.clone()
        call()
        assert torch.equal(first, out)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (192, 192), (256, 256), (512, 512), (128, 64), (192, 64), (256, 32), (128, 0),
                                     (72, 16), (120, 96), (8, 8), (136, 6), (100, 100), (66, 34), (3, 2), (1, 0), (40, 18), (328, 320)])
def test_shapes(name, layout, dim, rot):
    # rows a whole number of 16 bytes apart, or not
    for gap in (8, 3):
        check(name, [1, 17, 1000], [1, 5, 2], 7, 2, dim, rot, layout, seed=dim + rot, gap=gap)


@pytest.mark.parametrize("heads", [(1, 1), (32, 8), (5, 0), (0, 3), (64, 1), (33, 11)])
@pytest.mark.parametrize("dim", [64, 128, 192, 256, 100])
def test_heads(heads, dim):
    check("bf16", [9, 300], [3, 4], *heads, dim, dim // 2 // 16 * 16, "half", seed=2, gap=8)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("gap", [0, 3])
def test_without_norm_and_in_place(name, gap):
    check(name, [40], [40], 4, 2, 128, 128, "half", norm=False, seed=3, gap=gap)
    check(name, [40], [40], 4, 2, 128, 128, "half", place=True, seed=4, gap=gap)
    check(name, [40], [40], 4, 2, 192, 100, "interleaved", norm=False, place=True, seed=5, gap=gap)


@pytest.mark.parametrize("counts", [[0, 0, 4], [4, 0, 0, 3], [1] * 70, [0] * 40 + [5] + [0] * 40, [33, 1, 64]])
def test_ragged(counts):
    check("f16", [c + 7 * i for i, c in enumerate(counts)], counts, 2, 1, 128, 64, "half", seed=6)


def test_many_rows():
    # a warp takes several turns at a row's heads
    check("bf16", [9000] * 2, [1500] * 2, 32, 8, 128, 128, "half", even=True, seed=7, gap=8)
    check("bf16", [9000], [2000], 32, 8, 64, 64, "interleaved", even=True, seed=8, gap=8)
    check("f32", [9000], [1200], 24, 8, 256, 128, "half", even=True, seed=9, gap=8)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_rows_of_odd_channels(layout):
    # heads that do not come in pieces of eight: several of a row to a warp
    check("bf16", [9000] * 2, [700] * 2, 12, 3, 128, 36, layout, even=True, seed=16, gap=3)
    check("f32", [9000], [900], 10, 5, 200, 34, layout, even=True, seed=17)
    check("f16", [9000], [400], 30, 7, 65, 20, layout, even=True, seed=18)


@pytest.mark.parametrize("gap", [8, 3])
def test_one_side_normed(gap):
    # weights for the queries alone, or for the keys alone
    x = torch.randn(6, 3 * 128 + gap, generator=gen(19), device="cuda").to(torch.bfloat16)
    q, k = x[:, :256].unflatten(1, (2, 128)), x[:, 256:384].unflatten(1, (1, 128))
    w = (1 + torch.randn(128, generator=gen(20), device="cuda")).to(torch.bfloat16)
    lens = torch.tensor([77], dtype=torch.int32, device="cuda")
    freq, _ = frequencies(128)
    pos = positions([77], [6])
    for qw, kw in ((w, None), (None, w)):
        qo, ko = torch.empty(6, 2, 128, dtype=x.dtype, device="cuda"), torch.empty(6, 1, 128, dtype=x.dtype, device="cuda")
        g.gemv_qk_norm_rope("bf16", q, k, qo, ko, qw, kw, freq, lens, None, 1, 6, 2, 1, 128, 128)
        close("bf16", qo, *reference(q, qw, pos, freq, 128, "half", 1e-6, 1.0))
        close("bf16", ko, *reference(k, kw, pos, freq, 128, "half", 1e-6, 1.0))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout):
    # an angle's product in fp32 would be off by whole radians here
    check("f32", [131072, 1 << 20, (1 << 31) - 1, 5], [3, 2, 4, 5], 2, 1, 128, 128, layout, norm=False, factor=1.0, seed=10)


def test_frequencies_of_any_size():
    # zero, tiny, subnormal, one, negative and large ones
    f = torch.tensor([0.0, 1e-44, 1e-30, -0.3, 1.0, 3.5, 1000.25, 2.0 ** 20 + 0.5], device="cuda")
    x = torch.randn(6, 1, 16, generator=gen(11), device="cuda")
    lens = torch.tensor([(1 << 22) + 6], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    g.gemv_qk_norm_rope("f32", x, None, out, None, None, None, f, lens, None, 1, 6, 1, 0, 16, 16, layout="interleaved")
    y, m = reference(x, None, positions([(1 << 22) + 6], [6]), f, 16, "interleaved", 0.0, 1.0)
    # the fp64 product is exact to 2^-53 of an angle of 2^42; the kernel's to 2^-40 2^20 2^22 2^-22: below 2^-11 for the last
    bad = torch.tensor([2.0 ** -23] * 7 + [2.0 ** -9], dtype=torch.float64, device="cuda").repeat_interleave(2)
    assert bool(((out.double() - y).abs() <= (REL + bad) * m + 2.0 ** -24 * y.abs()).all())


def test_rows_that_no_sequence_has_stay():
    # rows before the first and behind the last, and a sequence with fewer tokens than rows
    x = torch.randn(20, 4, 128, generator=gen(12), device="cuda").to(torch.bfloat16)
    for place in (False, True):
        y = x.clone()
        out = None if place else torch.full_like(x, 5.0)
        lens = torch.tensor([9, 1, 0, 30], dtype=torch.int32, device="cuda")
        starts = torch.tensor([2, 5, 8, 8, 15], dtype=torch.int32, device="cuda")
        freq, _ = frequencies(128)
        g.gemv_qk_norm_rope("bf16", y, None, out, None, None, None, freq, lens, starts, 4, 20, 4, 0, 128, 128)
        got, old = (y, x) if place else (out, torch.full_like(x, 5.0))
        kept = [0, 1, 5, 6, 7, 15, 16, 17, 18, 19]
        assert torch.equal(got[kept], old[kept])
        pos = torch.tensor([6, 7, 8] + list(range(23, 30)), dtype=torch.float64, device="cuda")
        rows = [2, 3, 4] + list(range(8, 15))
        close("bf16", got[rows], *reference(x[rows], None, pos, freq, 128, "half", 0.0, 1.0))
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(128, 64), (24, 10)])
def test_specials_stay_in_their_pair(layout, dim, rot):
    x = torch.randn(3, 1, dim, generator=gen(13), device="cuda")
    x[0, 0, rot], x[0, 0, dim - 1] = math.nan, math.inf    # channels that do not turn
    x[1, 0, 0] = math.nan
    x[2, 0, 1] = -math.inf
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    freq, _ = frequencies(rot)
    out = torch.empty_like(x)
    g.gemv_qk_norm_rope("f32", x, None, out, None, None, None, freq, lens, None, 1, 3, 1, 0, dim, rot, layout=layout)
    y, m = reference(x, None, positions([50], [3]), freq, rot, layout, 0.0, 1.0)
    fine = torch.isfinite(y)
    assert torch.equal(torch.isfinite(out), fine)
    close("f32", out[fine], y[fine], m[fine])
    # with a norm, the head's mean takes them in
    w = torch.ones(dim, device="cuda")
    g.gemv_qk_norm_rope("f32", x, None, out, None, w, None, freq, lens, None, 1, 3, 1, 0, dim, rot, layout=layout)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[1]).all())


def test_zero_rows_and_epsilon():
    x = torch.zeros(2, 1, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    lens = torch.tensor([2], dtype=torch.int32, device="cuda")
    freq, _ = frequencies(64)
    g.gemv_qk_norm_rope("f32", x, None, None, None, w, None, freq, lens, None, 1, 2, 1, 0, 64, 64)
    assert bool((x == 0).all())
    g.gemv_qk_norm_rope("f32", x, None, None, None, w, None, freq, lens, None, 1, 2, 1, 0, 64, 64, eps=0.0)
    assert bool(torch.isnan(x).all())      # 0 / 0


def test_another_stream_and_a_replayed_graph():
    x = torch.randn(8, 3, 128, generator=gen(14), device="cuda").to(torch.bfloat16)
    w = (1 + torch.randn(128, generator=gen(15), device="cuda")).to(torch.bfloat16)
    lens = torch.full((8,), 20, dtype=torch.int32, device="cuda")
    freq, _ = frequencies(128)
    out = torch.empty_like(x)
    run = lambda stream=None: g.gemv_qk_norm_rope("bf16", x[:, :2], x[:, 2:], out[:, :2], out[:, 2:], w, w, freq, lens, None, 8, 8, 2, 1,  # noqa: E731
                                                  128, 128, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(s)
    s.synchronize()
    pos = torch.full((8,), 19.0, dtype=torch.float64, device="cuda")
    close("bf16", out, *reference(x, w, pos, freq, 128, "half", 1e-6, 1.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in (1, 2):
        lens += 100      # lengths live on the device: a replay turns by the new positions
        graph.replay()
        torch.cuda.synchronize()
        close("bf16", out, *reference(x, w, pos + 100 * step, freq, 128, "half", 1e-6, 1.0))


def two_pi(bits):
    """2 pi x 2^bits, a whole number: 32 atan(1/5) - 8 atan(1/239)."""
    def atan(n):
        total, term, k = 0, (1 << bits + 32) // n, 0
        while term:
            total += (-1) ** k * term // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    return 32 * atan(5) - 8 * atan(239) >> 32


def test_angles_to_the_last_position():
    # Angles good to 2^-23 for any frequency below 2^24 at any position, against whole numbers: a
    # pair (1, 0) becomes (cos, sin), each of which sincospif gives to one unit in the last place,
    # 2^-23 of it at most
    f = torch.tensor([0.75, 1.0, -3.5, 513.0625, 1000.25, 2.0 ** 20 + 0.5, -(2.0 ** 23 - 0.5), 2.0 ** 24 - 1], device="cuda")
    for last in ((1 << 31) - 1, (1 << 30) + 77, (1 << 22) + 6):
        x = torch.zeros(9, 1, 16, device="cuda")
        x[..., 0::2] = 1
        lens = torch.tensor([last], dtype=torch.int32, device="cuda")
        g.gemv_qk_norm_rope("f32", x, None, None, None, None, None, f, lens, None, 1, 9, 1, 0, 16, 16, layout="interleaved")
        for r, row in enumerate(x[:, 0].tolist()):
            for i, v in enumerate(f.tolist()):
                num, den = v.as_integer_ratio()
                turns = ((last - 9 + r) * num << 400) // (den * two_pi(200))     # x 2^200
                t = (turns & (1 << 200) - 1) / (1 << 200) * 2 * math.pi
                for got, want in ((row[2 * i], math.cos(t)), (row[2 * i + 1], math.sin(t))):
                    assert abs(got - want) <= 2.0 ** -23 * (1 + abs(want)), (v, last, r, got - want)
