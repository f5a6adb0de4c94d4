"""The 8-bit cache of keys and values: gemv_kv8_append against its definition, value by
value, and gemv_kv8_attention against a softmax in 64 bits over the cached values.

Tolerances.  The append is exact arithmetic (scales are powers of two, one rounding to
e4m3): equal bytes.  The attention: with w the softmax weights and v the values, the
weights are rounded to fp16 (2^-11 each), and the logits carry fp32 rounding and that of
q to fp16 after scaling by a power of two (2^-12 of each q element at most, where q is
fp16 or bf16: none, but for elements below 2^-28 of the row's largest): an error of d in
the logits changes the output by at most 2 d sum w |v|.  fp32 sums of D products, the
scale factors and exp2 give d <= (D + 8) 2^-23 max |scale q . k| terms, summed as
magnitudes.  So |err| <= (2^-11 + 2^-20 + 2 d) sum w |v| + u |out|, u the output type's
unit roundoff.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E4M3 = torch.float8_e4m3fn
BLOCK = 64


@pytest.fixture(autouse=True)
def _clean():
    g.test_stall(False)
    g.device_status()
    yield
    g.test_stall(False)
    g.device_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Cache:
    """A pool with a few blocks to spare, and sequences with their blocks scattered over
    it; all bytes are random at first, NaN among them, and the scales powers of two."""

    def __init__(self, lens, heads, dim, seed, width=None, spare=3):
        r = gen(seed)
        need = [-(-n // BLOCK) for n in lens]
        self.width = max(1, max(need, default=0)) if width is None else width
        self.pool = sum(need) + spare
        order = torch.randperm(self.pool, generator=r, device="cuda").tolist()
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for b in range(n):
                self.table[s, b] = order.pop()
        self.table = self.table.cuda()
        self.heads, self.dim, self.S = heads, dim, len(lens)
        self.k = torch.randint(0, 256, (self.pool, heads, BLOCK, dim), generator=r, device="cuda").to(torch.uint8)
        self.v = torch.randint(0, 256, (self.pool, heads, dim, BLOCK), generator=r, device="cuda").to(torch.uint8)
        self.ks = torch.exp2(torch.randint(-9, -5, (self.pool, heads), generator=r, device="cuda").float())
        self.vs = torch.exp2(torch.randint(-9, -5, (self.pool, heads), generator=r, device="cuda").float())
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def fill(self, seed):
        """Values as a cache holds them, in the tokens that the sequences have."""
        r = gen(seed)
        for s, n in enumerate(self.lens.tolist()):
            for b in range(-(-n // BLOCK)):
                c, pb = min(BLOCK, n - b * BLOCK), int(self.table[s, b])
                self.k[pb, :, :c] = (torch.randn(self.heads, c, self.dim, generator=r, device="cuda") * 100).to(E4M3).view(torch.uint8)
                self.v[pb, :, :, :c] = (torch.randn(self.heads, self.dim, c, generator=r, device="cuda") * 100).to(E4M3).view(torch.uint8)
        return self

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table


# ------------------------------------------------------------------ append
def power(a):
    if a == 0:
        return 2.0 ** -126
    m, e = math.frexp(a)   # a = m 2^e, 448 = 0.875 * 2^9
    return 2.0 ** max(-126, e - 9 + (m > 0.875))


def to8(x):
    return x.clamp(-448, 448).to(E4M3).view(torch.uint8)


def append_reference(c, k, v, starts):
    """The definition, block by block, on the cache's tensors as they were."""
    lens = c.lens.tolist()
    out = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    for s in range(c.S):
        n = starts[s + 1] - starts[s]
        before = lens[s] - n
        if n <= 0 or before < 0:
            continue
        for b in range(before // BLOCK, -(-lens[s] // BLOCK)):
            pb = int(c.table[s, b]) if b < c.width else -1
            if not 0 <= pb < c.pool:
                continue
            lo, hi = max(before, b * BLOCK) - b * BLOCK, min(lens[s] - b * BLOCK, BLOCK)
            first = starts[s] + b * BLOCK + lo - before
            for new, buf, sc, rows in ((k, out[0], out[2], True), (v, out[1], out[3], False)):
                for h in range(c.heads):
                    x = new[first:first + hi - lo, h].float()
                    fin = x[torch.isfinite(x)].abs()
                    scale = power(float(fin.max()) if fin.numel() else 0.0)
                    view = buf[pb, h] if rows else buf[pb, h].t()
                    if lo:
                        old = float(sc[pb, h])
                        scale = max(scale, old)
                        if scale != old:
                            view[:lo] = to8(view[:lo].contiguous().view(E4M3).float() * (old / scale))
                    view[lo:hi] = to8(x * (1.0 / scale))
                    sc[pb, h] = scale
    return out


def same_bytes(a, b):
    # e4m3's two NaN patterns are one value
    a, b = a.clone(), b.clone()
    a[a == 0xFF] = 0x7F
    b[b == 0xFF] = 0x7F
    return torch.equal(a, b)


def check_append(c, name, k, v, counts, even=False):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    want = append_reference(c, k, v, starts)
    st = None if even else torch.tensor(starts, dtype=torch.int32, device="cuda")
    g.gemv_kv8_append(name, *c.args(), k, v, c.lens, st, c.S, starts[-1])
    torch.cuda.synchronize()
    assert torch.equal(c.ks, want[2]) and torch.equal(c.vs, want[3])
    assert same_bytes(c.k, want[0]) and same_bytes(c.v, want[1])
    return want


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_append_one_token(name, dim):
    lens = [1, 2, 63, 64, 65, 128, 129, 200]
    c = Cache(lens, 3, dim, seed=dim).fill(1)
    x = torch.randn(len(lens), 6 * dim, generator=gen(2), device="cuda")
    x[::2] *= 20   # some raise their block's scale, some do not
    x = x.to(TYPES[name])
    # keys and values are columns of one tensor
    check_append(c, name, x[:, :3 * dim].view(-1, 3, dim), x[:, 3 * dim:].view(-1, 3, dim), [1] * len(lens), even=True)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("counts,lens", [
    ([5, 0, 64, 1, 63], [5, 70, 64, 65, 130]),       # ends and starts of blocks
    ([200, 3, 1, 130], [200, 66, 1, 140]),           # several blocks
    ([0, 0, 7], [0, 64, 100]),                        # sequences that get nothing
])
def test_append_ragged(name, counts, lens):
    c = Cache(lens, 2, 128, seed=3).fill(4)
    N = sum(counts)
    k = torch.randn(N, 2, 128, generator=gen(5), device="cuda").to(TYPES[name])
    v = (torch.randn(N, 2, 128, generator=gen(6), device="cuda") * 3).to(TYPES[name])
    check_append(c, name, k, v, counts)


@pytest.mark.parametrize("T", [3, 64, 65, 100])
def test_append_even(T):
    lens = [T, T + 1, T + 63, T + 64]
    c = Cache(lens, 1, 64, seed=T).fill(7)
    k = torch.randn(4 * T, 1, 64, generator=gen(8), device="cuda").to(torch.bfloat16)
    check_append(c, "bf16", k, k * 2, [T] * 4, even=True)


def test_append_specials():
    lens = [3, 66, 70]
    c = Cache(lens, 2, 64, seed=9).fill(10)
    k = torch.randn(6, 2, 64, generator=gen(11), device="cuda")
    v = torch.randn(6, 2, 64, generator=gen(12), device="cuda")
    k[0, 0, 5], k[1, 1, 6], v[2, 0, 7] = math.inf, -math.inf, math.nan
    k[3], v[3] = 0, 0
    v[4] = math.inf
    k[5] = 1e-38
    k[2, 0] = 448.0
    check_append(c, "f32", k, v, [3, 2, 1])


def test_append_unaligned_rows():
    # rows that start anywhere: element loads
    lens = [70, 40]
    c = Cache(lens, 1, 64, seed=13).fill(14)
    buf = torch.randn(50 * 131 + 3, generator=gen(15), device="cuda").to(torch.bfloat16)
    rows = buf[3:3 + 50 * 131].view(50, 131)
    k, v = rows[:, 1:65].view(50, 1, 64), rows[:, 66:130].view(50, 1, 64)
    check_append(c, "bf16", k, v, [20, 30])


def test_append_again_changes_nothing():
    lens = [100, 30]
    c = Cache(lens, 2, 128, seed=16).fill(17)
    k = (torch.randn(12, 2, 128, generator=gen(18), device="cuda") * 9).to(torch.bfloat16)
    want = check_append(c, "bf16", k, k, [4, 8])
    g.gemv_kv8_append("bf16", *c.args(), k, k, c.lens, torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda"), 2, 12)
    assert torch.equal(c.ks, want[2]) and same_bytes(c.k, want[0]) and same_bytes(c.v, want[1])


def test_append_where_the_cache_has_no_block():
    lens = [65, 10, 2]
    c = Cache(lens, 1, 64, seed=19).fill(20)
    c.table[0, 1] = -1            # no block for the last token
    c.table[1, 0] = c.pool        # past the pool
    c.lens[2] = 1                 # fewer tokens than new ones
    k = torch.randn(6, 1, 64, generator=gen(21), device="cuda").to(torch.bfloat16)
    check_append(c, "bf16", k, k, [2, 2, 2])
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)
    assert g.device_status() == (0, 0)


def test_append_token_by_token_is_append_at_once():
    """Scales are powers of two: moving a block to a larger one is exact (normal values)."""
    c1, c2 = Cache([150], 2, 128, seed=22), Cache([150], 2, 128, seed=22)
    # e4m3's subnormals: none of these is below 2^-14 of the largest of its block
    k = torch.randn(150, 2, 128, generator=gen(23), device="cuda").sign() * (0.02 + torch.rand(150, 2, 128, generator=gen(24), device="cuda"))
    k = (k * torch.linspace(0.5, 4, 150, device="cuda")[:, None, None]).to(torch.bfloat16)
    one = torch.tensor([0], dtype=torch.int32, device="cuda")
    for t in range(150):
        g.gemv_kv8_append("bf16", *c1.args(), k[t:t + 1], k[t:t + 1], one + t + 1, None, 1, 1)
    g.gemv_kv8_append("bf16", *c2.args(), k, k, c2.lens, None, 1, 150)
    assert torch.equal(c1.ks, c2.ks) and torch.equal(c1.vs, c2.vs)
    assert same_bytes(c1.k, c2.k) and same_bytes(c1.v, c2.v)


# ------------------------------------------------------------------ attention
def visible(n, T, t, window, sinks):
    i = n - T + t
    j = torch.arange(max(0, i + 1), device="cuda")
    if window:
        j = j[(i - j < window) | (j < sinks)]
    return j


def attention_reference(c, q, scale, window, sinks):
    """(out, lse, bound without the output's rounding), in 64 bits."""
    S, T, Hq, D = q.shape
    G = Hq // c.heads
    out = torch.zeros(S, T, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.full((S, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    cap = c.width * BLOCK
    for s, n in enumerate(c.lens.tolist()):
        n = min(max(n, 0), cap)
        for t in range(T):
            j = visible(n, T, t, window, sinks)
            if not j.numel():
                continue
            blk = c.table[s, j // BLOCK].long()
            ok = (blk >= 0) & (blk < c.pool)
            j, blk = j[ok], blk[ok]
            if not j.numel():
                continue
            for h in range(c.heads):
                k = c.k[blk, h, j % BLOCK].view(E4M3).float().double() * c.ks[blk, h, None].double()
                v = c.v[blk, h, :, j % BLOCK].contiguous().view(E4M3).float().double() * c.vs[blk, h, None].double()
                x = q[s, t, h * G:(h + 1) * G].double() * scale
                logits = x @ k.t()
                d = (D + 8) * 2.0 ** -23 * (x.abs() @ k.abs().t()).amax(-1, keepdim=True)
                w = torch.softmax(logits, -1)
                lse[s, t, h * G:(h + 1) * G] = torch.logsumexp(logits, -1)
                out[s, t, h * G:(h + 1) * G] = w @ v
                tol[s, t, h * G:(h + 1) * G] = (2.0 ** -11 + 2.0 ** -20 + 2 * d) * (w @ v.abs())
    return out, lse, tol


def attend(c, q, scale, window=0, sinks=0, stream=None, want_lse=True):
    S, T, Hq, D = q.shape
    name = "bf16" if q.dtype == torch.bfloat16 else "f16"
    out = torch.full((S, T, Hq, D), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((S, T, Hq), 5.0, device="cuda") if want_lse else None
    g.gemv_kv8_attention(name, *c.args(), q, c.lens, out, lse, S, T, Hq, scale, window=window, sinks=sinks, stream=stream)
    return out, lse


def check_attention(c, q, window=0, sinks=0, scale=None):
    scale = 1.0 / math.sqrt(c.dim) if scale is None else scale
    out, lse = attend(c, q, scale, window, sinks)
    ref, ref_lse, tol = attention_reference(c, q, scale, window, sinks)
    u = ROUND["bf16" if q.dtype == torch.bfloat16 else "f16"]
    # (a few of the cached values are NaN: beyond e4m3's range)
    fine, known = ~torch.isnan(ref), ~torch.isnan(ref_lse)
    assert torch.equal(~torch.isnan(out), fine) and torch.equal(~torch.isnan(lse), known)
    err, bound = (out.double() - ref)[fine].abs(), (tol + u * ref.abs() + 2.0 ** -24)[fine]
    assert bool((err <= bound).all()), float((err / bound).max())
    none = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, none) and bool((out[none] == 0).all())
    # the logits' error, and fp32 sums and logarithm
    e = (lse.double() - ref_lse)[known & ~none].abs()
    assert bool((e <= 1e-4 + 1e-6 * ref_lse[known & ~none].abs()).all()), float(e.max())
    out2, lse2 = attend(c, q, scale, window, sinks)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)), "two identical calls differ"
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32)), "two identical calls differ"
    return out, lse


def queries(c, T, group, seed, dtype=torch.bfloat16):
    return torch.randn(c.S, T, c.heads * group, c.dim, generator=gen(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 4, 7, 8, 9, 16, 33])
def test_attention_shapes(dim, group):
    c = Cache([1, 63, 64, 65, 300, 0, 1000], 2, dim, seed=dim + group).fill(30)
    check_attention(c, queries(c, 1, group, 31, torch.float16 if group % 2 else torch.bfloat16))
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("T,group", [(2, 1), (3, 4), (4, 6), (8, 8), (16, 1), (64, 2), (5, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_drafted(T, group, dim):
    # several queries, shorter sequences than queries among them: some see nothing
    c = Cache([0, 1, T - 1, T, T + 1, 64 + T, 200, 511], 1, dim, seed=T).fill(32)
    check_attention(c, queries(c, T, group, 33))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 130, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 65, 200])
def test_attention_window(window, sinks):
    lens = [1, 64, 65, 129, 200, 511, 1500]
    c = Cache(lens, 2, 64, seed=window + sinks).fill(34)
    for T in (4, 1):
        # blocks that no query sees are given back: their entries point nowhere
        for s, n in enumerate(lens):
            for b in range(c.width):
                if b * BLOCK >= sinks and (b + 1) * BLOCK <= n - T + 1 - window:
                    c.table[s, b] = -1
        check_attention(c, queries(c, T, 3, 35), window, sinks)
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("T", [1, 3])
def test_attention_unseen_values_are_anything(T):
    """NaN in keys and values that a query does not see leaves it untouched; a query that
    sees one gets NaN."""
    c = Cache([200, 40], 1, 128, seed=36).fill(37)
    q = queries(c, T, 2, 38)
    window, sinks, scale = 50, 2, 0.1
    ref, _ = check_attention(c, q, window, sinks, scale)
    for s, n in enumerate([200, 40]):
        for j in range(n):
            seen = [j <= n - T + t and (n - T + t - j < window or j < sinks) for t in range(T)]
            if not any(seen):
                c.k[int(c.table[s, j // BLOCK]), 0, j % BLOCK] = 0x7F
                c.v[int(c.table[s, j // BLOCK]), 0, :, j % BLOCK] = 0xFF
    out, _ = attend(c, q, scale, window, sinks)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    # the last token's value: seen by the last query alone
    c.v[int(c.table[0, 199 // BLOCK]), 0, 5, 199 % BLOCK] = 0x7F
    out, _ = attend(c, q, scale, window, sinks)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[0, T - 1, :, 5] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], ref[~want])


@pytest.mark.parametrize("dim,T,group,window,sinks", [
    (64, 4, 6, 0, 0), (64, 4, 6, 70, 3), (64, 8, 4, 0, 0), (64, 64, 1, 30, 0), (64, 3, 4, 65, 1),   # two to four row tiles, several items
    (128, 4, 4, 0, 0), (128, 8, 4, 100, 2), (192, 3, 5, 64, 0), (256, 5, 2, 0, 0)])
@pytest.mark.parametrize("longest", [180, 700])   # one launch, and items in parts
def test_attention_values_that_some_queries_see(dim, T, group, window, sinks, longest):
    """NaN in tokens that the later queries see and the earlier do not, or (with a window) the
    other way round: each query's result has it or is untouched, whatever row tile it is in."""
    lens = [longest, longest - 63, T]
    c = Cache(lens, 2, dim, seed=81).fill(82)
    c.k &= 0x77
    c.v &= 0xF7
    q = queries(c, T, group, 83)
    ref, ref_lse = check_attention(c, q, window, sinks, 0.1)
    want = torch.zeros_like(ref, dtype=torch.bool)
    for s, n in enumerate(lens):
        # a drafted token; and one that leaves the first queries' windows
        for j, ch in ((n - T + T // 2, 5), (n - T + T // 2 - window, dim - 1)):
            if not 0 <= j < n or (ch != 5 and not window):
                continue
            c.v[int(c.table[s, j // BLOCK]), 1, ch, j % BLOCK] = 0xFF
            for t in range(T):
                if bool((visible(n, T, t, window, sinks) == j).any()):
                    want[s, t, group:, ch] = True
    assert bool(want.any()) and not bool(want[:, :, group:, 5].all())
    out, lse = attend(c, q, 0.1, window, sinks)
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], ref[~want]) and torch.equal(lse, ref_lse)
    # a key: the whole result of the queries that see it
    j = longest - T + T // 2
    c.k[int(c.table[0, j // BLOCK]), 0, j % BLOCK, 3] = 0x7F
    out, lse = attend(c, q, 0.1, window, sinks)
    for t in range(T):
        if bool((visible(longest, T, t, window, sinks) == j).any()):
            want[0, t, :group] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], ref[~want])


def test_attention_large_and_small_logits():
    c = Cache([500, 90], 2, 64, seed=39).fill(40)
    for factor in (1e-6, 30.0, 3e3):
        check_attention(c, queries(c, 1, 4, 41, torch.bfloat16) * factor, scale=0.05)
    q = queries(c, 1, 4, 42)
    q[0, 0, 0] = 0     # equal weights
    q[1, 0, 3] *= torch.logspace(-6, 3, 64, device="cuda")   # elements far apart
    check_attention(c, q)


def test_attention_scales_apart():
    """Blocks whose scales differ by many orders, keys and values."""
    c = Cache([640], 1, 128, seed=43).fill(44)
    pb = c.table[0, :10].long()
    c.vs[pb, 0] = torch.exp2(torch.tensor([-30., 0, -12, 9, -60, 3, -9, -100, 20, -5], device="cuda"))
    c.ks[pb, 0] = torch.exp2(torch.tensor([-9., -20, -7, -8, -40, -8, -9, -120, -10, -6], device="cuda"))
    check_attention(c, queries(c, 2, 4, 45))


@pytest.mark.parametrize("lens,dim,T,group", [([1, 200], 128, 1, 4), ([1000, 64], 64, 1, 8), ([900, 70], 192, 3, 4), ([300], 256, 1, 2)])
def test_attention_large_and_small_values(lens, dim, T, group):
    """Values up to 7.8e34, a thousand of them: the largest sum of weighted values there can be is
    7.8e37.  And a power of two in the values' scales is one in the output, bit for bit (nothing
    here gets subnormal)."""
    c = Cache(lens, 2, dim, seed=70)
    c.k &= 0x77
    c.v &= 0xF7   # (both signs, at most 240, no NaN)
    q = queries(c, T, group, 71)
    vs = torch.exp2(torch.randint(-9, -5, c.vs.shape, generator=gen(72), device="cuda").float())
    c.vs = vs
    want, want_lse = check_attention(c, q, scale=0.05)
    for e in (114, -60):
        c.vs = vs * 2.0 ** e
        out, lse = check_attention(c, q, scale=0.05)
        assert torch.equal(out.float(), want.float() * 2.0 ** e) and torch.equal(lse, want_lse)
    # one visible value near the end of bf16's range
    c.lens[:] = 1
    c.vs = torch.full_like(vs, 2.0 ** 119)
    c.v[:] = 0x7E
    assert bool((attend(c, q[:, :1].contiguous(), 0.05)[0].float() == 448 * 2.0 ** 119).all())


def test_attention_strided_queries():
    c = Cache([100, 77, 300], 2, 64, seed=46).fill(47)
    wide = torch.randn(3, 2, 8 * 64 + 256, generator=gen(48), device="cuda").to(torch.bfloat16)
    q = wide[:, :, 64:64 + 8 * 64].view(3, 2, 8, 64)
    got, _ = attend(c, q, 0.125)
    want, _ = check_attention(c, q.contiguous(), scale=0.125)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    odd = torch.randn(3 * 2 * 515 + 1, generator=gen(49), device="cuda").to(torch.float16)[1:].view(3, 2, 515)[:, :, 2:514]
    got, _ = attend(c, odd.view(3, 2, 8, 64), 0.125)
    want, _ = check_attention(c, odd.contiguous().view(3, 2, 8, 64), scale=0.125)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("lens", [[20000], [1] * 700, [0, 0, 9000, 0, 3, 0], list(range(1, 400, 3)), [0, 0, 0]])
def test_attention_work_shares(lens):
    """One long sequence, many short ones, empty ones between: items that many CTAs
    share, and CTAs that have many items."""
    c = Cache(lens, 2, 64, seed=50)
    # (random bytes, without NaN)
    c.k &= 0x77
    c.v &= 0x77
    check_attention(c, queries(c, 1, 2, 51))


# items in parts by the hundred and by the few: every width of the kernel that joins them
@pytest.mark.parametrize("lens,heads,dim,T,group,window,sinks", [
    ([30000], 1, 192, 1, 16, 0, 0), ([9001], 4, 128, 1, 4, 0, 0), ([7000], 2, 256, 1, 3, 0, 0), ([12000, 0, 5], 1, 64, 5, 5, 0, 0),
    ([2000] * 5 + [1, 0, 777], 4, 128, 1, 4, 0, 0), ([1000] * 16, 8, 128, 1, 4, 0, 0), ([3000] * 12, 4, 64, 4, 6, 1030, 4),
    ([900] * 40, 8, 64, 1, 8, 0, 0)])
def test_attention_joins(lens, heads, dim, T, group, window, sinks):
    c = Cache(lens, heads, dim, seed=60)
    c.k &= 0x77
    c.v &= 0x77
    check_attention(c, queries(c, T, group, 61), window, sinks)
    assert g.device_status() == (0, 0)


def test_attention_far_blocks():
    """A pool beyond 2^32 bytes, its last blocks in use."""
    blocks, heads, dim = 70000, 8, 128
    assert blocks * heads * BLOCK * dim > 2 ** 32
    c = Cache([130], heads, dim, seed=52)
    c.pool = blocks
    c.k = torch.zeros(blocks, heads, BLOCK, dim, dtype=torch.uint8, device="cuda")
    c.v = torch.zeros(blocks, heads, dim, BLOCK, dtype=torch.uint8, device="cuda")
    c.ks, c.vs = torch.ones(blocks, heads, device="cuda"), torch.ones(blocks, heads, device="cuda")
    c.table[0] = torch.tensor([blocks - 1, blocks - 3, 0], dtype=torch.int32)
    k = torch.randn(130, heads, dim, generator=gen(53), device="cuda").to(torch.bfloat16)
    g.gemv_kv8_append("bf16", *c.args(), k, k * 2, c.lens, None, 1, 130)
    check_attention(c, queries(c, 1, 4, 54))
    # the appended values are there: within e4m3's rounding
    got = c.v[blocks - 1, 3].view(E4M3).float() * c.vs[blocks - 1, 3]
    want = 2 * k[:64, 3].float().t()
    assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + c.vs[blocks - 1, 3] * 2.0 ** -10).all())


@pytest.mark.parametrize("window,first_seen", [(0, True), (2 ** 30 - 1, False), (2 ** 30, True), (2 ** 40, True)])
def test_attention_longest_table(window, first_seen):
    """2^30 tokens, in a pool of 4096 blocks that the table goes over again and again: the first
    token decides the result of a query that sees it (its weight is e^64 times another's)."""
    c = Cache([1], 1, 64, seed=80, width=2 ** 24)
    blocks = 4096
    c.k = torch.zeros(blocks, 1, BLOCK, 64, dtype=torch.uint8, device="cuda")
    c.v = torch.ones(blocks, 1, 64, BLOCK, device="cuda").to(E4M3).view(torch.uint8)
    c.ks, c.vs = torch.ones(blocks, 1, device="cuda"), torch.ones(blocks, 1, device="cuda")
    c.table[0] = torch.arange(2 ** 24, dtype=torch.int32, device="cuda") % (blocks - 1) + 1
    c.table[0, 0] = 0
    one, three = (int(torch.tensor(f).to(E4M3).view(torch.uint8)) for f in (1.0, 3.0))
    c.k[0, 0, 0], c.v[0, 0, :, 0] = one, three
    c.lens[:] = 2 ** 30
    out, lse = attend(c, torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda"), 1.0, window=window)
    assert bool((out == (3.0 if first_seen else 1.0)).all())
    # (equal weights: fp32 holds their sums to 2^-24 for each of the blocks that a warp adds, 14 k)
    want = 64.0 if first_seen else math.log(2 ** 30 - 1)
    assert abs(float(lse[0, 0, 0]) - want) <= 14000 * 2.0 ** -24 + 1e-5


def test_attention_where_the_cache_has_no_block():
    c = Cache([300, 100], 1, 64, seed=55).fill(56)
    c.table[0, 2] = -5
    c.table[0, 4] = c.pool
    check_attention(c, queries(c, 2, 4, 57))
    assert g.device_status() == (g.ERR_INVALID_VALUE, 64)
    c.lens[1] = 10 ** 9          # past the table
    c.table[1] = c.table[0]
    c.table[:, :] = c.table[0, 0]
    check_attention(c, queries(c, 1, 2, 58))
    c.lens[1] = -7
    check_attention(c, queries(c, 1, 2, 59))


def test_attention_on_a_stream_and_in_a_graph():
    c = Cache([3000, 5], 2, 128, seed=60).fill(61)
    q = queries(c, 1, 4, 62)
    want, want_lse = check_attention(c, q, scale=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = attend(c, q, 0.1, stream=s, want_lse=False)
    s.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemv_kv8_attention("bf16", *c.args(), q, c.lens, out, lse, 2, 1, 8, 0.1)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    # lengths are read on the device: a replay follows them
    c.lens[0] = 1000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), attend(c, q, 0.1)[0].view(torch.int16))


def test_bounded_wait():
    c = Cache([64], 1, 128, seed=63).fill(64)
    q = queries(c, 1, 4, 65)
    torch.cuda.synchronize()
    g.test_stall(True, 50_000_000)
    attend(c, q, 0.1)
    status, bits = g.device_status()
    assert status == g.ERR_DEVICE_TIMEOUT and bits & 16
    g.test_stall(False)
    check_attention(c, q, scale=0.1)
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("lens,heads,dim,T,group", [([3000, 40, 0, 700], 2, 128, 1, 4), ([900] * 300, 1, 64, 4, 6), ([20000], 1, 192, 1, 16)])
def test_bounded_wait_of_shared_items(lens, heads, dim, T, group):
    """Items in parts, and warps with several items, whose waits run out: the kernel that joins
    the parts finds what the scratch memory held before (here another call's sums)."""
    c = Cache(lens, heads, dim, seed=66)
    c.k &= 0x77
    c.v &= 0x77
    q = queries(c, T, group, 67)
    A = torch.full((12000, 4096), 0x38, dtype=torch.uint8, device="cuda").view(E4M3)   # shared tiles: fp32 sums in the pool
    x, ones = torch.full((3, 4096), 0x38, dtype=torch.uint8, device="cuda").view(E4M3), torch.ones(94, 32, device="cuda")
    g.gemv_f8(A, ones, x, ones[:3], None, torch.empty(3, 12000, dtype=torch.bfloat16, device="cuda"), 12000, 4096, 3)
    torch.cuda.synchronize()
    g.test_stall(True, 20_000_000)
    attend(c, q, 0.1)
    status, bits = g.device_status()
    assert status == g.ERR_DEVICE_TIMEOUT and bits & 16
    g.test_stall(False)
    check_attention(c, q, scale=0.1)
    assert g.device_status() == (0, 0)
