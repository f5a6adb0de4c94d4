"""gemv_kv8_prefix_attention at the ends of its ranges: logits far below zero, values of
the smallest scales, many groups, groups that share little.

Tolerances: those of tests/test_gpu_prefix.py.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g
from tests.test_gpu_kv8 import BLOCK, E4M3, ROUND, attend, attention_reference
from tests.test_gpu_prefix import Shared, call, check, queries, same, small_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    g.test_stall(False)
    g.device_status()
    yield
    assert g.device_status() == (0, 0)


def finite(c):
    """The cache without NaN: its largest value in their place."""
    for t in (c.k, c.v):
        t[(t & 0x7F) == 0x7F] = 0x7E
    return c


@pytest.mark.parametrize("far", [100.0, 200.0, 1000.0])
@pytest.mark.parametrize("S,T,group", [(3, 1, 4), (3, 16, 4)])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_blocks_far_below(dim, S, T, group, far):
    # runs of blocks all of whose logits are near -far: the first ones; all but one in the middle, so
    # that every share of the work begins with such a block; all of them, the sequences' own too
    P = 1280
    lens = [P + T + 70 * i for i in range(S)]
    q = None
    for which in range(3):
        c = finite(Shared([0, S], [P], lens, 2, dim, seed=120 + dim).fill(121))
        if q is None:
            q = queries(c, T, group, 122)
            q[...] = q[:1, :1, :1]
        c.ks[:] = 2.0 ** -12
        if which == 0:
            blocks = c.table[0, :2].long()
        elif which == 1:
            blocks = torch.cat((c.table[0, :7], c.table[0, 8:P // BLOCK])).long()
        else:
            blocks = torch.arange(c.pool, device="cuda")
        q0 = q[0, 0, 0].float()
        c.k[blocks] = (q0 * -64).clamp(-448, 448).to(E4M3).view(torch.uint8)
        c.ks[blocks] = 2.0 ** -6
        out, lse = check(c, q, scale=far / float(q0.square().sum()))
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("power", [-126, -123, -118])
def test_the_smallest_value_scales(dim, power):
    # values that bf16 holds, 2^-120 and below: nothing on the way may flush them to zero.  To the
    # bounds of the other tests half of bf16's smallest step, 2^-134
    P = 1280
    c = finite(Shared([0, 4], [P], [P + 5, P + 70, P + 1, P + 130], 2, dim, seed=123).fill(124))
    c.vs[:] = 2.0 ** power
    q = queries(c, 2, 4, 125)
    scale = 1 / math.sqrt(dim)
    if dim % 128:      # logits whose rounding shows
        scale *= 30
    ref, _, tol = attention_reference(c, q, scale, 0, 0)
    tol = tol + small_weights(c, q, scale) + ROUND["bf16"] * ref.abs() + 2.0 ** -134
    assert float(ref.abs().amax()) > 2.0 ** (power + 3)
    for out in (call(c, q, scale)[0], attend(c, q, scale)[0]):
        err = (out.double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


def test_hundreds_of_groups():
    # most of them share nothing, in long runs: a CTA's share begins behind any number of groups
    G, n = 320, 3
    prefix = [64 * (1 + i % 5) + 9 if i % 40 in (0, 7, 39) or i > 300 else (0, 63, -1)[i % 3] for i in range(G)]
    lens = [max(prefix[i // n], 0) + 1 + i % 70 for i in range(n * G)]
    c = finite(Shared([n * i for i in range(G + 1)], prefix, lens, 1, 64, seed=129, width=200).fill(130))
    q = queries(c, 1, 16, 131)
    k = g.launch_count()
    call(c, q, 0.1)
    assert g.launch_count() - k == 3
    check(c, q)


def us(run, calls=5):
    """Least time of a call, of a few rounds of captured ones."""
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            run()
    best = math.inf
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


def test_a_thousand_groups_take_no_walk():
    # a CTA finds its share 32 groups at a time: one after the other they took 0.7 us each, three times
    # what gemv_kv8_attention takes for all of it
    G, n, P = 1024, 8, 512
    c = Shared([n * i for i in range(G + 1)], [P] * G, [0] * (n * G), 1, 64, seed=132, width=16)
    c.pool = G * 8 + n * G * 2
    c.k = torch.randint(0, 120, (c.pool, 1, BLOCK, 64), device="cuda", dtype=torch.uint8)
    c.v = torch.randint(0, 120, (c.pool, 1, 64, BLOCK), device="cuda", dtype=torch.uint8)
    c.ks = c.vs = torch.full((c.pool, 1), 2.0 ** -9, device="cuda")
    s = torch.arange(n * G, device="cuda")[:, None]
    c.table[:, :8] = (s // n * 8 + torch.arange(8, device="cuda")).int()
    c.table[:, 8:10] = (G * 8 + s * 2 + torch.arange(2, device="cuda")).int()
    c.lens.fill_(P + 100)
    q = torch.randn(n * G, 1, 16, 64, device="cuda").to(torch.bfloat16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    args = ("bf16", *c.args(), q, c.lens)
    shared = us(lambda: g.gemv_kv8_prefix_attention(*args, c.firsts, c.prefix, out, None, n * G, 1, 16, 0.125))
    apart = us(lambda: g.gemv_kv8_attention(*args, want, None, n * G, 1, 16, 0.125))
    assert bool(((out.float() - want.float()).abs() <= 2.0 ** -6 * want.float().abs() + 2.0 ** -8).all())
    assert shared < 2 * apart, (shared, apart)


@pytest.mark.parametrize("firsts", [[0, 1], [0, 1, 2, 3, 4], [0, 0, 0, 2, 4]])
def test_as_many_groups_as_sequences(firsts):
    # nothing is shared, or (groups without sequences) little: the call is passed on, with equal bits
    S = firsts[-1]
    c = Shared(firsts, [640] * S, [650 + 40 * i for i in range(S)], 2, 128, seed=126).fill(127)
    q = queries(c, 1, 4, 128)
    n = g.launch_count()
    out, lse = call(c, q, 0.1)
    assert g.launch_count() - n == 2
    want, want_lse = attend(c, q, 0.1)
    assert same(out, want) and same(lse, want_lse)


def wide(firsts, prefix, lens, heads, dim, seed):
    """Tables so wide that any groups of three sequences are shared."""
    return Shared(firsts, prefix, lens, heads, dim, seed, width=1 + 4_000_000_000 // (len(lens) * BLOCK * heads * dim * 2))


def shared(c, q, **k):
    """Checked, and not passed on."""
    n = g.launch_count()
    call(c, q, 0.1)
    assert g.launch_count() - n == 3
    return check(c, q, **k)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_sequence_to_a_group(dim):
    # its own queries share a sequence's blocks, where they are many
    for S, T in ((1, 64), (3, 17)):
        P = 2000
        c = wide(list(range(S + 1)), [P + 100 * i for i in range(S)], [P + 100 * i + T + 30 for i in range(S)], 1, dim, seed=151).fill(152)
        shared(c, queries(c, T, 4, 153), again=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups_of_every_kind(dim):
    # groups of one and many sequences, an empty one, sequences before the first and behind the last,
    # idle places, sequences shorter than the prefix, or by one token too short to see it whole
    firsts, prefix = [1, 2, 2, 9, 13, 14], [300, 640, 1000, 64, 500]
    lens = [333, 302, 1003, 1100, 0, 960 + 2, 960 + 1, 50, 1024, 66, 65, 64, 0, 600, 40, 0]
    c = wide(firsts, prefix, lens, 2, dim, seed=133).fill(134)
    shared(c, queries(c, 2, 3, 135, torch.float16))


def test_seventy_groups():
    n, G = 3, 70
    prefix = [64 * (i % 7) + 5 for i in range(G)]
    c = wide([n * i for i in range(G + 1)], prefix, [prefix[i // n] + 3 + i % 90 for i in range(n * G)], 1, 64, seed=136).fill(137)
    shared(c, queries(c, 1, 4, 138), again=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups_one_behind_the_other(dim):
    # calls of different work lists, back to back, as in tests/test_gpu_prefix.py
    c = wide([0, 5, 9], [1500, 3000], [1600 + 30 * i for i in range(5)] + [3001 + 70 * i for i in range(4)], 2, dim, seed=139).fill(140)
    kinds = [queries(c, 1, 4, 141), queries(c, 8, 4, 142), queries(c, 2, 8, 143)]
    try:
        g.set_launch_overlap("off")
        want = []
        for q in kinds:
            want.append(call(c, q, 0.1))
            torch.cuda.synchronize()
        for mode in ("launch", "weights"):
            g.set_launch_overlap(mode)
            n = g.launch_count()
            got = [call(c, kinds[i % 3], 0.1) for i in range(30)]
            assert g.launch_count() - n == 90
            torch.cuda.synchronize()
            for i, (out, lse) in enumerate(got):
                assert same(out, want[i % 3][0]) and same(lse, want[i % 3][1]), (mode, i)
    finally:
        g.set_launch_overlap("launch")


def test_a_sink_and_a_long_flat_rest():
    # one token far above all others, whose weights of 2^-20 count by their number
    P = 32768
    c = finite(Shared([0, 4], [P], [P + 5, P + 9, P + 1, P + 70], 1, 128, seed=144).fill(145))
    c.ks[:] = 2.0 ** -12
    b = int(c.table[0, 0])
    q = queries(c, 1, 4, 146)
    q[...] = q[:1, :, :1]                       # all alike, so that one key suits all
    c.k[b, 0, 7] = (q[0, 0, 0].float() * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)
    c.ks[b, 0] = 2.0 ** -6
    shared(c, q)


def test_scratch_memory_has_a_limit():
    # 512 groups of three sequences: a whole tile for each group and head would take 620 MB, the output
    # takes 13 MB.  Forty groups stay below the limit
    c = wide([3 * i for i in range(513)], [64] * 512, [65 + i % 5 for i in range(3 * 512)], 8, 128, seed=147)
    c.k[:], c.v[:] = 0x30, 0x38
    q = queries(c, 1, 4, 148)
    want = attend(c, q, 0.1)
    n = g.launch_count()
    out, lse = call(c, q, 0.1)
    assert g.launch_count() - n == 2
    assert same(out, want[0]) and same(lse, want[1])
    few = wide([3 * i for i in range(41)], [64] * 40, [65 + i % 5 for i in range(3 * 40)], 8, 128, seed=149)
    few.k[:], few.v[:] = 0x30, 0x38
    shared(few, queries(few, 1, 4, 150), again=False)
