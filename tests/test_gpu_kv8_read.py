"""gemv_kv8_read: cached tokens back as rows.

The value is exact arithmetic: e4m3 (exact in fp32) times a power of two, rounded once to
the output type.  So equal values, NaN for NaN.
"""
from __future__ import annotations

import pytest
import torch

import decode_linear_layers_gb300 as g
from tests.test_gpu_kv8 import BLOCK, E4M3, TYPES, Cache, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.device_status()


def reference(c, counts, dt, old_k, old_v):
    """The definition, token by token, over rows as they were."""
    k, v, row = old_k.clone(), old_v.clone(), 0
    ks, vs = c.ks.float(), c.vs.float()
    for s, n in enumerate(c.lens.tolist()):
        for i in range(counts[s]):
            pos = n - counts[s] + i
            pb = int(c.table[s, pos // BLOCK]) if n >= counts[s] and pos // BLOCK < c.width else -1
            if 0 <= pb < c.pool:
                k[row] = (c.k[pb, :, pos % BLOCK].view(E4M3).float() * ks[pb, :, None]).to(dt)
                v[row] = (c.v[pb, :, :, pos % BLOCK].contiguous().view(E4M3).float() * vs[pb, :, None]).to(dt)
            row += 1
    return k, v


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def check(c, name, counts, even=False, spare=2, width=None, first=0):
    dt, N, row = TYPES[name], sum(counts), c.heads * c.dim
    st = [0]
    for n in counts:
        st.append(st[-1] + n)
    starts = None if even else torch.tensor(st, dtype=torch.int32, device="cuda")
    rows = N + (0 if even else spare)     # rows behind the last sequence stay
    width = 2 * row + 8 if width is None else width
    buf = torch.full((rows * width + first,), 3.0, dtype=dt, device="cuda")
    mat = buf[first:first + rows * width].view(rows, width)
    k, v = mat[:, :row].unflatten(1, (c.heads, c.dim)), mat[:, row:2 * row].unflatten(1, (c.heads, c.dim))
    want = reference(c, counts, dt, k, v)
    g.gemv_kv8_read(name, *c.args(), k, v, c.lens, starts, c.S, rows)
    torch.cuda.synchronize()
    assert same(k, want[0]) and same(v, want[1])
    assert bool((mat[:, 2 * row:] == 3).all()) and bool((buf[:first] == 3).all())
    # one side alone: dense rows
    for side in (0, 1):
        one = torch.full((rows, c.heads, c.dim), 3.0, dtype=dt, device="cuda")
        g.gemv_kv8_read(name, *c.args(), one if side == 0 else None, one if side == 1 else None, c.lens, starts, c.S, rows)
        assert same(one, want[side])


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("heads", [1, 3])
def test_read_shapes(name, dim, heads):
    # every byte of the pool is random: NaN, subnormals and e4m3's largest among them
    c = Cache([1, 63, 64, 65, 200, 130], heads, dim, seed=dim + heads)
    check(c, name, [1, 63, 30, 65, 2, 100])


@pytest.mark.parametrize("counts,lens", [([5, 0, 64, 1, 63], [5, 70, 64, 65, 130]), ([200, 3, 1, 130], [200, 66, 1, 140]), ([0, 0, 7], [0, 64, 100])])
def test_read_ragged(counts, lens):
    check(Cache(lens, 2, 128, seed=3), "bf16", counts)


@pytest.mark.parametrize("T", [1, 3, 64, 65, 100])
def test_read_even(T):
    check(Cache([T, T + 1, T + 63, T + 64], 2, 64, seed=T), "f16", [T] * 4, even=True)


@pytest.mark.parametrize("name", TYPES)
def test_read_unaligned_rows(name):
    c = Cache([70, 40], 1, 64, seed=13)
    check(c, name, [20, 30], width=131, first=3)


def test_read_many_sequences():
    lens = [(37 * i) % 300 for i in range(150)]
    check(Cache(lens, 1, 64, seed=14), "bf16", [n // 2 for n in lens])


def test_read_where_the_cache_has_no_block():
    c = Cache([65, 10, 2, 192], 1, 64, seed=19, width=3)
    c.table[0, 1] = -1            # no block for the last token
    c.table[1, 0] = c.pool        # past the pool
    c.lens[2] = 1                 # fewer tokens than rows
    c.lens[3] = 700               # tokens beyond the table
    check(c, "bf16", [2, 2, 2, 600])
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("name", TYPES)
def test_read_gives_back_what_append_took(name):
    lens, counts = [40, 200, 64], [40, 150, 1]
    c = Cache(lens, 2, 128, seed=22).fill(23)
    k = torch.randn(191, 2, 128, generator=gen(24), device="cuda").to(TYPES[name])
    v = (torch.randn(191, 2, 128, generator=gen(25), device="cuda") * 5).to(TYPES[name])
    starts = torch.tensor([0, 40, 190, 191], dtype=torch.int32, device="cuda")
    g.gemv_kv8_append(name, *c.args(), k, v, c.lens, starts, 3, 191)
    got_k, got_v = torch.empty_like(k), torch.empty_like(v)
    g.gemv_kv8_read(name, *c.args(), got_k, got_v, c.lens, starts, 3, 191)
    for a, b in ((k, got_k), (v, got_v)):
        # half a step of e4m3: 2^-4 of the value, or of its smallest normal 2^-6 for those below it, at
        # a scale of at most twice the block's largest / 448; and the type's own rounding
        top = float(a.float().abs().max())
        assert bool(((a.float() - b.float()).abs() <= a.float().abs() * (2.0 ** -4 + 2.0 ** -8) + 2.0 ** -10 * 2 * top / 448).all())


def test_read_in_a_graph_on_a_stream():
    c = Cache([100, 30], 2, 128, seed=26).fill(27)
    k = torch.zeros(8, 2, 128, device="cuda")
    v = torch.zeros_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.gemv_kv8_read("f32", *c.args(), k, v, c.lens, None, 2, 8, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemv_kv8_read("f32", *c.args(), k, v, c.lens, None, 2, 8)
    c.lens -= 20
    graph.replay()
    torch.cuda.synchronize()
    want = reference(c, [4, 4], torch.float32, k, v)
    assert same(k, want[0]) and same(v, want[1])
