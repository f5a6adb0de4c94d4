"""gemv_kv8_prefix_attention against a softmax in 64 bits over the cached values.

Tolerance.  That of gemv_kv8_attention (tests/test_gpu_kv8.py: fp16 weights, fp32 logits,
sums and outputs), and for weights below fp16's normal range: half of fp16's smallest step,
2^-25, against 2^8 at least for the largest weight times its block's value scale.  Each of n
tokens is off by at most 2^-33 of that product, times an e4m3 value of at most 448: n 2^-33
times the largest w x scale, times 448.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g
from tests.test_gpu_kv8 import BLOCK, E4M3, ROUND, Cache, attention_reference, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    g.test_stall(False)
    g.device_status()
    yield
    g.test_stall(False)
    g.device_status()


class Shared(Cache):
    """Sequences of which those of a group begin with the same blocks.  The table is wide
    enough for the blocks to be shared (short ones are passed on to gemv_kv8_attention);
    entries behind a sequence's own are -1."""

    def __init__(self, firsts, prefix, lens, heads, dim, seed, width=None):
        if width is None:
            width = 1 + max([320_000_000 // (len(lens) * BLOCK * heads * dim * 2)] + [-(-n // BLOCK) for n in lens])
        super().__init__(lens, heads, dim, seed, width)
        for i, p in enumerate(prefix):
            n = min(max(p, 0) // BLOCK, self.width)
            long = [s for s in range(firsts[i], firsts[i + 1]) if lens[s] >= n * BLOCK]
            for s in long:
                self.table[s, :n] = self.table[long[0], :n]
        self.firsts = torch.tensor(firsts, dtype=torch.int32, device="cuda")
        self.prefix = torch.tensor(prefix, dtype=torch.int32, device="cuda")


def call(c, q, scale, firsts=True, stream=None, want_lse=True, fill=5.0):
    S, T, Hq, D = q.shape
    name = "bf16" if q.dtype == torch.bfloat16 else "f16"
    out = torch.full((S, T, Hq, D), fill, dtype=q.dtype, device="cuda")
    lse = torch.full((S, T, Hq), fill, device="cuda") if want_lse else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    g.gemv_kv8_prefix_attention(name, *c.args(), q, c.lens, c.firsts if firsts else None, c.prefix, out, lse, S, T, Hq, scale,
                                stream=stream)
    return out, lse


def same(a, b):
    """Equal bits (a few of the cached values are NaN: beyond e4m3's range)."""
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def small_weights(c, q, scale):
    """n 2^-33 448 (largest w x value scale) for each row, in 64 bits."""
    S, T, Hq, D = q.shape
    G = Hq // c.heads
    out = torch.zeros(S, T, Hq, 1, dtype=torch.float64, device="cuda")
    for s, n in enumerate(c.lens.tolist()):
        n = min(n, c.width * BLOCK)
        for t in range(T):
            i = n - T + t + 1
            if i <= 0:
                continue
            j = torch.arange(i, device="cuda")
            blk = c.table[s, j // BLOCK].long()
            ok = (blk >= 0) & (blk < c.pool)
            j, blk = j[ok], blk[ok]
            if not j.numel():
                continue
            for h in range(c.heads):
                k = c.k[blk, h, j % BLOCK].view(E4M3).double() * c.ks[blk, h, None].double()
                w = torch.softmax(q[s, t, h * G:(h + 1) * G].double() * scale @ k.t(), -1) * c.vs[blk, h].double()
                out[s, t, h * G:(h + 1) * G, 0] = i * 2.0 ** -33 * 448 * w.amax(-1)
    return out


def check(c, q, scale=None, firsts=True, again=True):
    scale = 1.0 / math.sqrt(c.dim) if scale is None else scale
    out, lse = call(c, q, scale, firsts)
    ref, ref_lse, tol = attention_reference(c, q, scale, 0, 0)
    tol = tol + small_weights(c, q, scale)
    u = ROUND["bf16" if q.dtype == torch.bfloat16 else "f16"]
    fine, known = ~torch.isnan(ref), ~torch.isnan(ref_lse)
    assert torch.equal(~torch.isnan(out), fine) and torch.equal(~torch.isnan(lse), known)
    err, bound = (out.double() - ref)[fine].abs(), (tol + u * ref.abs() + 2.0 ** -24)[fine]
    assert bool((err <= bound).all()), float((err / bound).max())
    none = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, none) and bool((out[none] == 0).all())
    e = (lse.double() - ref_lse)[known & ~none].abs()
    assert bool((e <= 1e-4 + 1e-6 * ref_lse[known & ~none].abs()).all()), float(e.max())
    if again:
        out2, lse2 = call(c, q, scale, firsts)
        assert same(out, out2) and same(lse, lse2), "two identical calls differ"
    return out, lse


def queries(c, T, group, seed, dtype=torch.bfloat16):
    return torch.randn(c.S, T, c.heads * group, c.dim, generator=gen(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 4, 7, 16])
def test_shapes(dim, group):
    # one group; own tokens that end anywhere, none of them whole blocks among the first
    P = 700
    c = Shared([0, 5], [P], [P + 1, P + 64, P + 200, 641, P + 30], 2, dim, seed=dim + group).fill(30)
    check(c, queries(c, 1, group, 31, torch.float16 if group % 2 else torch.bfloat16), firsts=False)
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("S,T,group", [(3, 64, 1), (2, 64, 4), (9, 16, 2), (33, 2, 4), (1, 33, 4), (40, 1, 8)])
def test_rows_of_one_and_more_tiles(S, T, group, dim):
    # 132 to 512 rows: a set of tiles full, partly full, a last one of a few rows
    P = 576
    c = Shared([0, S], [P], [P + T + (37 * i) % 150 for i in range(S)], 1, dim, seed=S + T).fill(32)
    check(c, queries(c, T, group, 33), again=False)


@pytest.mark.parametrize("prefix", [0, -5, 1, 63, 64, 65, 127, 128, 320, 321, 1000000])
def test_prefix_lengths(prefix):
    lens = [prefix + 20 + i if 0 < prefix < 1000 else 400 + i for i in range(4)]
    for width in (None, 7):
        c = Shared([0, 4], [prefix], lens, 2, 128, seed=41, width=width).fill(42)
        check(c, queries(c, 2, 4, 43), firsts=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups(dim):
    # groups of one and many sequences, an empty one, sequences before the first and behind the last,
    # idle places, sequences shorter than the prefix, or by one token too short to see it whole
    firsts, prefix = [1, 2, 2, 9, 13, 14], [300, 640, 1000, 64, 500]
    lens = [333, 302, 1003, 1100, 0, 960 + 2, 960 + 1, 50, 1024, 66, 65, 64, 0, 600, 40, 0]
    c = Shared(firsts, prefix, lens, 2, dim, seed=44 + dim).fill(45)
    check(c, queries(c, 2, 3, 46, torch.float16))
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("idle", [1, 5, 40])
def test_idle_places_before_the_others(idle):
    # the first places of a group are idle, and what their tables hold is no block
    P = 1000
    lens = [0] * idle + [P + 9, P + 80, P + 2] + [0] * idle + [P + 30]
    n = idle + 3
    c = Shared([0, n, 2 * idle + 4], [P, P], lens, 2, 128, seed=110).fill(111)
    c.table[:idle] = c.pool + 5
    c.table[n:n + idle] = -7
    check(c, queries(c, 1, 4, 112))
    assert g.device_status() == (0, 0)


def test_no_one_shares():
    c = Shared([0, 4], [100000], [300, 70, 0, 641], 2, 128, seed=113).fill(114)
    check(c, queries(c, 3, 4, 115))
    assert g.device_status() == (0, 0)


def test_many_groups():
    G = 70
    firsts = [2 * i for i in range(G + 1)]
    prefix = [64 * (i % 7) + 5 for i in range(G)]
    c = Shared(firsts, prefix, [prefix[i // 2] + 3 + i % 90 for i in range(2 * G)], 1, 64, seed=47).fill(48)
    check(c, queries(c, 1, 4, 49), again=False)


@pytest.mark.parametrize("dim", [128, 192])
def test_a_long_prefix(dim):
    P = 20000
    c = Shared([0, 6], [P], [P + 3 + 50 * i for i in range(6)], 2, dim, seed=50).fill(51)
    check(c, queries(c, 1, 4, 52))
    check(c, queries(c, 16, 4, 53, torch.float16), again=False)


def test_a_batch_of_decode_size():
    P = 4096
    c = Shared([0, 64], [P], [P + 1 + 13 * i for i in range(64)], 8, 128, seed=54).fill(55)
    check(c, queries(c, 1, 4, 56), again=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_of_very_different_size(dim):
    P = 1280
    c = Shared([0, 3], [P], [P + 70] * 3, 2, dim, seed=57).fill(58)
    for kind in range(4):
        r = gen(59 + kind)
        if kind == 0:      # values: any size, some blocks all zeros with the smallest scale
            c.vs = torch.exp2(torch.randint(-30, 20, (c.pool, 2), generator=r, device="cuda").float())
            c.v[c.table[0, 3].long()] = 0
            c.vs[c.table[0, 3].long()] = 2.0 ** -126
        elif kind == 1:    # rising along the sequence, logits too: the reference moves at every block
            step = torch.arange(P // BLOCK, device="cuda").float()
            c.vs[c.table[0, :P // BLOCK].long()] = torch.exp2(2 * step - 20)[:, None]
            c.ks[c.table[0, :P // BLOCK].long()] = torch.exp2(0.25 * step - 9).log2().round().exp2()[:, None]
        elif kind == 2:    # falling
            step = torch.arange(P // BLOCK, device="cuda").float()
            c.vs[c.table[0, :P // BLOCK].long()] = torch.exp2(20 - 2 * step)[:, None]
        else:              # large logits: softmax picks single tokens
            c.vs[:] = 0.25
            c.ks[:] = 2.0 ** -3
        check(c, queries(c, 1, 4, 63))


def test_large_logits_with_values_of_zero():
    # a block of zeros (the smallest scale) has the largest logits by far: its weights are all that
    # counts in the sums, and P cannot hold them beside the other values'
    P = 1280
    c = Shared([0, 3], [P], [P + 70] * 3, 2, 128, seed=116).fill(117)
    q = queries(c, 1, 4, 118)
    q[...] = q[:1, :, :1]
    for at, far in ((0, 60.0), (0, 140.0), (5, 60.0), (5, 140.0), (19, 300.0)):
        d = Shared([0, 3], [P], [P + 70] * 3, 2, 128, seed=116).fill(117)
        b = d.table[0, at].long()
        d.v[b], d.vs[b] = 0, 2.0 ** -126
        norm = float(q[0, 0, 0].float().square().sum())
        d.k[b] = (q[0, 0, 0].float() * 64).clamp(-448, 448).to(E4M3).view(torch.uint8)   # all 64 tokens alike
        d.ks[b] = 2.0 ** -6
        check(d, q, scale=far / norm * math.log(2.0))


def test_a_sink_and_a_long_flat_rest():
    # one token far above all others, whose weights of 2^-20 count by their number
    P = 32768
    c = Shared([0, 2], [P], [P + 5, P + 9], 1, 128, seed=64).fill(65)
    c.ks[:] = 2.0 ** -12
    b = int(c.table[0, 0])
    q = queries(c, 1, 4, 66)
    q[...] = q[:1, :, :1]                       # all alike, so that one key suits all
    c.k[b, 0, 7] = (q[0, 0, 0].float() * 100).clamp(-448, 448).to(E4M3).view(torch.uint8)
    c.ks[b, 0] = 2.0 ** -6
    check(c, q)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0, 1e-30])
def test_scale(scale):
    c = Shared([0, 4], [500], [520, 501, 600, 513], 2, 128, seed=67).fill(68)
    check(c, queries(c, 1, 4, 69), scale=scale)


def test_queries_of_any_size():
    c = Shared([0, 4], [500], [520, 501, 600, 513], 1, 128, seed=70).fill(71)
    q = queries(c, 1, 4, 72).float()
    q *= torch.exp2(torch.arange(16, device="cuda").float() * 4 - 40).view(4, 1, 4, 1)
    check(c, q.to(torch.bfloat16), scale=1.0)


def test_what_no_query_sees_has_no_influence():
    # bytes behind the sequences' ends are NaN; so are other blocks of the pool
    lens = [650, 641, 700, 0, 100]
    c = Shared([0, 5], [640], lens, 2, 128, seed=73).fill(74)
    c2 = Shared([0, 5], [640], lens, 2, 128, seed=73)
    c2.k[:], c2.v[:] = 0x7F, 0xFF
    for s, n in enumerate(lens):
        for b in range(-(-n // BLOCK)):
            pb, m = int(c.table[s, b]), min(BLOCK, n - b * BLOCK)
            c2.k[pb, :, :m], c2.v[pb, :, :, :m] = c.k[pb, :, :m], c.v[pb, :, :, :m]
    c2.ks[:], c2.vs[:] = c.ks, c.vs
    q = queries(c, 2, 4, 75)
    a, b = call(c, q, 0.1), call(c2, q, 0.1)
    assert same(a[0], b[0]) and same(a[1], b[1])


def test_nan_that_is_seen():
    c = Shared([0, 3], [640], [650, 641, 700], 1, 128, seed=76).fill(77)
    c.v[int(c.table[0, 2]), 0, 5, 9] = 0x7F
    q = queries(c, 1, 4, 78)
    out, _ = call(c, q, 0.1)
    assert bool(torch.isnan(out[..., 5]).all()) and int(torch.isnan(out).sum()) == out[..., 5].numel()
    c.k[int(c.table[0, 1]), 0, 3, 0] = 0x7F      # a key: all of the row
    out, lse = call(c, q, 0.1)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_a_query_of_infinities_and_nan():
    c = Shared([0, 3], [640], [650, 641, 700], 1, 128, seed=79).fill(80)
    q = queries(c, 1, 4, 81)
    want, _ = call(c, q, 0.1)
    q[1, 0, 2, 3], q[2, 0, 0, 7] = math.nan, math.inf
    out, _ = call(c, q, 0.1)
    for s in range(3):
        for h in range(4):
            if (s, h) in ((1, 2), (2, 0)):
                assert bool((torch.isnan(out[s, 0, h]) | (out[s, 0, h] == 0)).all())
            else:
                assert same(out[s, 0, h], want[s, 0, h])


@pytest.mark.parametrize("gap,first", [(8, 0), (3, 1)])
def test_strided_queries(gap, first):
    c = Shared([0, 4], [500], [520, 501, 600, 513], 2, 128, seed=82).fill(83)
    q = queries(c, 2, 4, 84)
    width = 8 * 128 + gap
    buf = torch.zeros(8 * width + first, dtype=torch.bfloat16, device="cuda")
    rows = buf[first:].view(8, width)[:, :8 * 128]
    rows.copy_(q.view(8, -1))
    view = rows.unflatten(1, (8, 128)).unflatten(0, (4, 2))
    a, b = call(c, q, 0.1), call(c, view, 0.1)
    assert same(a[0], b[0]) and same(a[1], b[1])
    none = call(c, view, 0.1, want_lse=False)
    assert same(a[0], none[0])


def test_blocks_outside_the_pool():
    c = Shared([0, 3], [640], [650, 700, 645], 2, 128, seed=85).fill(86)
    c.table[:, 4] = -1
    c.table[:, 7] = c.pool
    check(c, queries(c, 1, 4, 87), again=False)
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)
    c.table[:] = -1
    out, lse = call(c, queries(c, 1, 4, 88), 0.1)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_what_is_passed_on(dim):
    # the same results to rounding, from gemv_kv8_attention's kernels or from the shared ones
    lens = [700, 800, 701]
    narrow = Shared([0, 3], [640], lens, 2, dim, seed=89, width=13).fill(90)
    wide = Shared([0, 3], [640], lens, 2, dim, seed=89).fill(90)
    q = queries(narrow, 1, 4, 91)
    for c, launches in ((narrow, 2), (wide, 3)):
        n = g.launch_count()
        call(c, q, 0.1)
        assert g.launch_count() - n == launches
        check(c, q)


def test_lengths_beyond_the_table():
    c = Shared([0, 3], [640], [704, 704, 700], 2, 128, seed=95).fill(96)
    c.lens[0] = 64 * c.width + 5000        # counts as the table's size
    check(c, queries(c, 1, 4, 97), again=False)
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)      # its table has no blocks there


def test_alone_and_in_a_group_of_other_size():
    # what a sequence gets differs only by rounding where the group around it changes
    P = 1000
    c = Shared([0, 8], [P], [P + 5 + i for i in range(8)], 2, 128, seed=98).fill(99)
    q = queries(c, 1, 4, 100)
    check(c, q)
    for n in (1, 3):
        d = Shared([0, n], [P], [P + 5 + i for i in range(n)], 2, 128, seed=98)
        d.k, d.v, d.ks, d.vs, d.pool = c.k, c.v, c.ks, c.vs, c.pool
        d.table[:, :20] = c.table[:n, :20]
        check(d, q[:n])


def test_graphs_that_run_at_once():
    P = 2000
    c = Shared([0, 8], [P], [P + 5 + 20 * i for i in range(8)], 2, 128, seed=101).fill(102)
    q1, q2 = queries(c, 1, 4, 103), queries(c, 4, 4, 104)
    want1, want2 = call(c, q1, 0.1), call(c, q2, 0.1)
    outs, graphs = [], []
    for q in (q1, q2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(c, q, 0.1))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (out, lse), (want, wl) in zip(outs, (want1, want2)):
        assert same(out, want) and same(lse, wl)
    # the lengths, and the prefix, are read at each replay
    c.lens += 40
    c.prefix.fill_(1500)
    graphs[0].replay()
    torch.cuda.synchronize()
    again = call(c, q1, 0.1)
    assert same(outs[0][0], again[0]) and same(outs[0][1], again[1])


def test_on_two_streams():
    P = 3000
    c = Shared([0, 8], [P], [P + 5 + 20 * i for i in range(8)], 2, 64, seed=105).fill(106)
    q = queries(c, 2, 4, 107)
    want = call(c, q, 0.1)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [call(c, q, 0.1, stream=streams[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    for out, lse in got:
        assert same(out, want[0]) and same(lse, want[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_calls_one_behind_the_other(dim):
    # calls of different work lists, back to back: each kernel may begin before the one ahead of it
    # is done, and the scratch memory is the same
    c = Shared([0, 5, 9], [1500, 3000], [1600 + 30 * i for i in range(5)] + [3001 + 70 * i for i in range(4)], 2, dim, seed=108).fill(109)
    kinds = [queries(c, 1, 4, 110), queries(c, 8, 4, 111), queries(c, 2, 8, 112)]
    try:
        g.set_launch_overlap("off")
        want = []
        for q in kinds:
            want.append(call(c, q, 0.1))
            torch.cuda.synchronize()
        for mode in ("launch", "weights"):
            g.set_launch_overlap(mode)
            got = [call(c, kinds[i % 3], 0.1) for i in range(30)]
            torch.cuda.synchronize()
            for i, (out, lse) in enumerate(got):
                assert same(out, want[i % 3][0]) and same(lse, want[i % 3][1]), (mode, i)
    finally:
        g.set_launch_overlap("launch")


def test_a_block_that_stands_in_a_table_twice():
    c = Shared([0, 4], [700], [705 + 40 * i for i in range(4)], 2, 128, seed=113).fill(114)
    c.table[:, 3] = c.table[0, 1]      # among the shared blocks
    c.table[2, 11] = c.table[2, 0]     # a shared one among a sequence's own
    check(c, queries(c, 2, 4, 115), firsts=False)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_a_wait_that_runs_out(dim):
    c = Shared([0, 4], [5000], [5005 + i for i in range(4)], 2, dim, seed=108).fill(109)
    q = queries(c, 1, 4, 110)
    want = call(c, q, 0.1)
    torch.cuda.synchronize()
    g.test_stall(1, 20_000_000)
    call(c, q, 0.1)
    status, bits = g.device_status()
    assert status == g.ERR_DEVICE_TIMEOUT and bits & 16
    g.test_stall(0)
    again = call(c, q, 0.1)
    assert g.device_status() == (0, 0)
    assert same(again[0], want[0]) and same(again[1], want[1])
