"""Operators of a served batch around the 8-bit cache, as measured cases.

Three operators that stand between the QKV projection and the output projection, beside
the append to the 8-bit cache and the attention over it: the norm of each head of the
queries and keys with the rotation by their positions (``rope``), the cached keys and
values of a range of tokens read back (``read``), and the attention of sequences that
share a long prefix, whose blocks meet all of their queries at once (``prefix``).

``run`` computes them in their plain form with elementary torch operations, in 32 bits
(angles in 64) and rounded once (``own`` false), or calls the library (``own`` true).
``exact`` is the definition in 64 bits.

8-bit values are e4m3 (torch.float8_e4m3fn).
"""
import math

import torch

own = False

BLOCK = 64    # tokens of the cache per block
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of a layer with 32 query and 8 key heads: latency
        {"name": "rope_token", "op": "rope", "type": "bf16", "S": 1, "T": 1, "ragged": False, "q_heads": 32, "k_heads": 8,
         "dim": 128, "rot": 128, "layout": "half", "norm": True, "longest": 1000},
        # one token for each sequence of a decode batch
        {"name": "rope_batch", "op": "rope", "type": "bf16", "S": 64, "T": 1, "ragged": False, "q_heads": 32, "k_heads": 8,
         "dim": 128, "rot": 128, "layout": "half", "norm": True, "longest": 8192},
        # prompts of different lengths, 15 k tokens in all: bytes
        {"name": "rope_prompt", "op": "rope", "type": "bf16", "S": 5, "T": 4096, "ragged": True, "q_heads": 32, "k_heads": 8,
         "dim": 128, "rot": 128, "layout": "half", "norm": True, "longest": 9000},
        # neighbouring channels, a third of the head, no norm, an odd number of tokens far out
        {"name": "rope_far", "op": "rope", "type": "f32", "S": 1, "T": 1023, "ragged": False, "q_heads": 7, "k_heads": 1,
         "dim": 192, "rot": 64, "layout": "interleaved", "norm": False, "longest": 131072},
        # a short conversation moved out: latency
        {"name": "read_short", "op": "read", "type": "bf16", "S": 1, "T": 100, "ragged": False, "heads": 8, "dim": 128,
         "longest": 100},
        # the last tokens of a batch, any place in a block, for a layer that works in 32 bits
        {"name": "read_window", "op": "read", "type": "f32", "S": 24, "T": 500, "ragged": False, "heads": 4, "dim": 64,
         "longest": 20000},
        # what is cached of several prompts, for a chunk's attention in 16 bits
        {"name": "read_prompt", "op": "read", "type": "f16", "S": 5, "T": 9000, "ragged": True, "heads": 8, "dim": 128,
         "longest": 9000},
        # one long sequence: bytes
        {"name": "read_long", "op": "read", "type": "bf16", "S": 1, "T": 131072, "ragged": False, "heads": 8, "dim": 128,
         "longest": 131072},
        # a few samples of one short prompt: latency
        {"name": "prefix_short", "op": "prefix", "type": "bf16", "groups": 1, "S": 4, "T": 1, "heads": 8, "group": 4,
         "dim": 128, "prefix": 1000, "longest": 100, "idle": 0},
        # a decode batch behind one long document
        {"name": "prefix_batch", "op": "prefix", "type": "bf16", "groups": 1, "S": 64, "T": 1, "heads": 8, "group": 4,
         "dim": 128, "prefix": 32768, "longest": 1024, "idle": 0},
        # four drafted tokens for each sequence, three documents, idle places in the batch
        {"name": "prefix_drafted", "op": "prefix", "type": "f16", "groups": 3, "S": 24, "T": 4, "heads": 4, "group": 6,
         "dim": 64, "prefix": 20000, "longest": 500, "idle": 2},
        # questions of 64 tokens about one document, all at once: arithmetic
        {"name": "prefix_chunk", "op": "prefix", "type": "bf16", "groups": 1, "S": 16, "T": 64, "heads": 8, "group": 4,
         "dim": 128, "prefix": 16384, "longest": 200, "idle": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "read", "prefix", "prefix"])
    dim = rng.choice([64, 128, 128, 192, 256])
    if op == "rope":
        k_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        S, kind = _spread(rng, 1, 96), rng.choice(["bf16", "f16", "f32"])
        row = (1 + group) * k_heads * dim * (2 if kind == "f32" else 1)
        T = rng.choice([1, 1, 4, _spread(rng, 1, 4096)])
        T = max(1, min(T, 60_000_000 // (S * row)))
        return {"op": op, "type": kind, "S": S, "T": T, "ragged": rng.random() < 0.5, "q_heads": k_heads * group,
                "k_heads": k_heads, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                "layout": rng.choice(["half", "interleaved"]), "norm": rng.random() < 0.6,
                "longest": max(T, _spread(rng, 1, 131072))}
    heads = rng.choice([1, 2, 4, 8])
    if op == "read":
        S, kind = _spread(rng, 1, 96), rng.choice(["bf16", "f16", "f32"])
        longest = max(1, min(_spread(rng, 1, 131072), 134_000_000 // (S * heads * dim * (2 if kind == "f32" else 1))))
        return {"op": op, "type": kind, "S": S, "T": min(longest, rng.choice([longest, _spread(rng, 1, 4096)])),
                "ragged": rng.random() < 0.5, "heads": heads, "dim": dim, "longest": longest}
    groups = rng.choice([1, 1, 2, 5])
    S, T, group = groups + _spread(rng, 1, 96) - 1, rng.choice([1, 1, 1, 2, 4, 16, 64]), rng.choice([1, 2, 3, 4, 6, 8, 16])
    rows = S * T * heads * group * dim
    prefix = max(1, min(_spread(rng, 1, 65536), 60_000_000_000 // rows, 134_000_000 // (groups * heads * dim)))
    return {"op": op, "type": rng.choice(["bf16", "f16"]), "groups": groups, "S": S, "T": T, "heads": heads, "group": group,
            "dim": dim, "prefix": prefix, "longest": max(T, min(_spread(rng, 1, 2048), 100_000_000 // (S * heads * dim))),
            "idle": rng.choice([0, 0, 1]) if S > groups else 0}


# ------------------------------------------------------------------ inputs
def _lengths(n, longest, least=1):
    """Spread over [least, longest], the first the longest."""
    return [max(least, math.ceil(longest * (1.0 - (i * 0.6180339887) % 1.0))) for i in range(n)]


def _counts(case):
    """Tokens asked for of each sequence: T, or spread over [0, T] where ragged."""
    lens = _lengths(case["S"], case["longest"])
    n = [case["T"] if not case["ragged"] else int(case["T"] * (1.0 - (i * 0.3819660113) % 1.0)) for i in range(case["S"])]
    return [min(a, b) for a, b in zip(n, lens)]


def _shape(case):
    """A batch behind shared prefixes: (first sequence of each group and S, prefix of each
    group, tokens of each sequence with its prefix; an idle place has none)."""
    P, S = case["groups"], case["S"]
    first = [i * S // P for i in range(P + 1)]
    prefix = _lengths(P, case["prefix"])
    own_tokens = _lengths(S, case["longest"], case["T"])
    lens = []
    for g in range(P):
        lens += [prefix[g] + own_tokens[s] for s in range(first[g], first[g + 1])]
    for i in range(case["idle"]):
        lens[S - 1 - i] = 0
    return first, prefix, lens


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _power(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))


def _pool(gen, blocks, H, D):
    """Blocks of keys (blocks x heads x BLOCK x dim), of values (blocks x heads x dim x
    BLOCK), and their scales (blocks x heads), as the cache holds them."""
    k = torch.empty(blocks, H, BLOCK, D, dtype=torch.uint8, device="cuda")
    v = torch.empty(blocks, H, D, BLOCK, dtype=torch.uint8, device="cuda")
    ks, vs = torch.empty(blocks, H, device="cuda"), torch.empty(blocks, H, device="cuda")
    for lo in range(0, blocks, 512):
        n = min(512, blocks - lo)
        level = torch.exp(0.3 * _rand(gen, n, H, 1, 1))
        for buf, sc, shape, c in ((k, ks, (n, H, BLOCK, D), 1.5), (v, vs, (n, H, D, BLOCK), 0.7)):
            x = _rand(gen, *shape) * level * c
            s = _power(x.abs().amax(dim=(2, 3)))
            buf[lo:lo + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            sc[lo:lo + n] = s
    return k, v, ks, vs


def _stale(gen, k, v, table, lens):
    """The last block of each sequence: bytes past its tokens are what was there before."""
    S, H, D = len(lens), k.shape[1], k.shape[3]
    some = [s for s in range(S) if lens[s] % BLOCK]
    if not some:
        return
    rest = torch.tensor([lens[s] % BLOCK for s in some], device="cuda")
    pb = table[some, torch.tensor([lens[s] // BLOCK for s in some], device="cuda")].long()
    old = torch.arange(BLOCK, device="cuda")[None] >= rest[:, None]
    junk = torch.randint(0, 256, (len(some), H, BLOCK, D), generator=gen, device="cuda").to(torch.uint8)
    k[pb] = torch.where(old[:, None, :, None], junk, k[pb])
    v[pb] = torch.where(old[:, None, None, :], junk.transpose(2, 3), v[pb])


def _table(gen, rows, spare=3):
    """A table out of each sequence's block numbers, scattered over a pool with a few
    blocks to spare; -1 behind them."""
    pool = max([max(r) + 1 for r in rows if r], default=0) + spare
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(len(r) for r in rows))
    place = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int64, device="cuda")
    return torch.where(place >= 0, order[place.clamp_min(0)], torch.full_like(order[:1], -1)), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dtype, D = case["op"], TYPES[case["type"]], case["dim"]
    st = dict(case)
    if op == "rope":
        Q, K, S = case["q_heads"], case["k_heads"], case["S"]
        counts, lens = _counts(case), _lengths(case["S"], case["longest"])
        N = sum(counts)
        # queries, keys and values are columns of the fused projection's output
        st["qkv"] = _rand(gen, N, (Q + 2 * K) * D).mul_(1.0 + torch.rand(N, 1, generator=gen, device="cuda")).to(dtype)
        st["q"], st["k"] = st["qkv"][:, :Q * D].unflatten(1, (Q, D)), st["qkv"][:, Q * D:(Q + K) * D].unflatten(1, (K, D))
        st["turned"] = torch.empty(N, (Q + K) * D, dtype=dtype, device="cuda")
        st["q_out"] = st["turned"][:, :Q * D].unflatten(1, (Q, D))
        st["k_out"] = st["turned"][:, Q * D:].unflatten(1, (K, D))
        for name in ("q_weight", "k_weight"):
            st[name] = (1.0 + 0.3 * _rand(gen, D)).to(dtype) if case["norm"] else None
        # frequencies of a context stretched four times
        st["inv_freq"] = (0.25 * 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) * 2 / case["rot"])).float().cuda()
        st["factor"] = 1.0 + 0.1 * math.log(4.0)
        even = all(n == case["T"] for n in counts)
        st["N"], st["starts"] = N, None if even else torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda")
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return st
    H = case["heads"]
    if op == "read":
        counts, lens = _counts(case), _lengths(case["S"], case["longest"])
        N, rows, at = sum(counts), [], 0
        for n, c in zip(lens, counts):  # blocks before the tokens asked for were given back
            gone, held = (n - c) // BLOCK, -(-n // BLOCK)
            rows.append([-1] * gone + list(range(at, at + held - gone)))
            at += held - gone
        st["table"], pool = _table(gen, rows)
        st["k"], st["v"], st["k_scale"], st["v_scale"] = _pool(gen, pool, H, D)
        _stale(gen, st["k"], st["v"], st["table"].clamp_min(0), lens)
        st["new_k"], st["new_v"] = (torch.empty(N, H, D, dtype=dtype, device="cuda") for _ in range(2))
        even = all(n == case["T"] for n in counts)
        st["N"], st["starts"] = N, None if even else torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda")
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return st
    S, T, G = case["S"], case["T"], case["group"]
    first, prefix, lens = _shape(case)
    rows, at = [], 0
    for g in range(case["groups"]):
        common = list(range(at, at + prefix[g] // BLOCK))  # whole blocks are shared
        at += len(common)
        for s in range(first[g], first[g + 1]):
            more = max(0, -(-lens[s] // BLOCK) - len(common))
            rows.append(common + list(range(at, at + more)) if lens[s] else [])
            at += more
    st["table"], pool = _table(gen, rows)
    st["k"], st["v"], st["k_scale"], st["v_scale"] = _pool(gen, pool, H, D)
    _stale(gen, st["k"], st["v"], st["table"], lens)
    st["q"] = _rand(gen, S, T, H * G, D).to(dtype)
    st["out"] = torch.empty(S, T, H * G, D, dtype=dtype, device="cuda")
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    st["firsts"] = None if case["groups"] == 1 else torch.tensor(first, dtype=torch.int32, device="cuda")
    st["shape"] = (first, prefix, max(lens))  # the plain form's sizes
    return st


# ------------------------------------------------------------------ plain forms
def _positions(st):
    """(sequence, position) of each of the N rows."""
    S, N, lens = st["S"], st["N"], st["lens"].long()
    i = torch.arange(N, device="cuda")
    starts = torch.arange(S + 1, device="cuda") * (N // S) if st["starts"] is None else st["starts"].long()
    seq = torch.searchsorted(starts, i, right=True) - 1
    return seq, lens[seq] - starts[seq + 1] + i


def _plain_rope(st):
    _, pos = _positions(st)
    r, inter = st["rot"] // 2, st["layout"] == "interleaved"
    angle = pos[:, None].double() * st["inv_freq"].double()
    cos, sin = ((f(angle) * st["factor"]).float()[:, None] for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (x[..., 0:2 * r:2], x[..., 1:2 * r:2]) if inter else (x[..., :r], x[..., r:2 * r])
        a, b = a * cos - b * sin, b * cos + a * sin
        both = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
        return torch.cat((both, x[..., 2 * r:]), -1).to(TYPES[st["type"]])

    return [turned(st["q"], st["q_weight"]), turned(st["k"], st["k_weight"])]


def _plain_read(st):
    seq, pos = _positions(st)
    blk, slot = st["table"][seq, pos // BLOCK].long(), pos % BLOCK
    out = []
    for buf, sc in ((st["k"].transpose(1, 2), st["k_scale"]), (st["v"].permute(0, 3, 1, 2), st["v_scale"])):
        x = buf[blk, slot].view(torch.float8_e4m3fn).float()
        out.append((x * sc[blk][:, :, None]).to(TYPES[st["type"]]))
    return out


def _taken(st, tab):
    """Keys (... x heads x tokens x dim) and values (... x heads x dim x tokens) in 32 bits."""
    H, D, tab = st["heads"], st["dim"], tab.long().clamp_min(0)
    k = st["k"][tab].view(torch.float8_e4m3fn).float() * st["k_scale"][tab][..., None, None]
    v = st["v"][tab].view(torch.float8_e4m3fn).float() * st["v_scale"][tab][..., None, None]
    return (k.transpose(-4, -3).reshape(*tab.shape[:-1], H, tab.shape[-1] * BLOCK, D),
            v.movedim(-4, -2).reshape(*tab.shape[:-1], H, D, tab.shape[-1] * BLOCK))


def _plain_prefix(st):
    S, T, H, G, D = st["S"], st["T"], st["heads"], st["group"], st["dim"]
    first, prefix, most = st["shape"]
    q = (st["q"].float() * (1.0 / math.sqrt(D))).view(S, T, H, G, D)
    out = torch.empty(S, T, H, G, D, device="cuda")
    at = st["lens"].long()[:, None] - T + torch.arange(T, device="cuda")  # position of each query
    for g in range(st["groups"]):
        a, b = first[g], first[g + 1]
        n, P = b - a, prefix[g] // BLOCK
        if n == 0:
            continue
        W = max(P, min(-(-most // BLOCK), st["table"].shape[1]))
        seen = torch.arange(W * BLOCK, device="cuda") <= at[a:b, :, None]     # n x T x tokens
        kp, vp = _taken(st, st["table"][a, :P])                                # once for the group
        ko, vo = _taken(st, st["table"][a:b, P:W])
        some = seen[:, :, P * BLOCK:].any(1)                                   # what no query sees is nothing
        ko = torch.where(some[:, None, :, None], ko, torch.zeros_like(ko[:1, :1, :1, :1]))
        vo = torch.where(some[:, None, None, :], vo, torch.zeros_like(vo[:1, :1, :1, :1]))
        for h in range(H):
            qh = q[a:b, :, h].reshape(n * T * G, D)
            x = torch.cat(((qh @ kp[h].t()).view(n, T, G, -1), (qh.view(n, T * G, D) @ ko[:, h].transpose(1, 2)).view(n, T, G, -1)), -1)
            x = x.masked_fill(~seen[:, :, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
            total = p.sum(-1, keepdim=True)
            o = (p[..., :P * BLOCK].reshape(n * T * G, -1) @ vp[h].t()).view(n, T, G, D)
            o = o + (p[..., P * BLOCK:].reshape(n, T * G, -1) @ vo[:, h].transpose(1, 2)).view(n, T, G, D)
            out[a:b, :, h] = torch.where(total > 0, o / total, torch.zeros_like(o))
    return out.view(S, T, H * G, D).to(st["out"].dtype)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if not own:
        return {"rope": _plain_rope, "read": _plain_read, "prefix": _plain_prefix}[op](st)
    import decode_linear_layers_gb300 as g
    if op == "rope":
        g.gemv_qk_norm_rope(st["type"], st["q"], st["k"], st["q_out"], st["k_out"], st["q_weight"], st["k_weight"],
                            st["inv_freq"], st["lens"], st["starts"], st["S"], st["N"], st["q_heads"], st["k_heads"],
                            st["dim"], st["rot"], layout=st["layout"], eps=1e-6, factor=st["factor"])
        return [st["q_out"], st["k_out"]]
    cache = st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"]
    if op == "read":
        g.gemv_kv8_read(st["type"], *cache, st["new_k"], st["new_v"], st["lens"], st["starts"], st["S"], st["N"])
        return [st["new_k"], st["new_v"]]
    g.gemv_kv8_prefix_attention(st["type"], *cache, st["q"], st["lens"], st["firsts"], st["prefix_lens"], st["out"], None,
                                st["S"], st["T"], st["heads"] * st["group"], 1.0 / math.sqrt(st["dim"]))
    return st["out"]


# ------------------------------------------------------------------ bytes and operations
def work(case):
    op, size, D = case["op"], {"bf16": 2, "f16": 2, "f32": 4}[case["type"]], case["dim"]
    if op == "rope":
        n = sum(_counts(case))
        heads = n * (case["q_heads"] + case["k_heads"])
        return {"bytes": 2 * size * heads * D + (2 * size * D if case["norm"] else 0) + 2 * case["rot"] + 4 * case["S"],
                "flops": heads * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    H = case["heads"]
    if op == "read":
        lens, counts = _lengths(case["S"], case["longest"]), _counts(case)
        n = sum(counts)
        blocks = sum(-(-a // BLOCK) - (a - c) // BLOCK for a, c in zip(lens, counts) if c)
        return {"bytes": 2 * n * H * D * (1 + size) + blocks * (8 * H + 4), "flops": 2 * n * H * D}
    T, G = case["T"], case["group"]
    first, prefix, lens = _shape(case)
    keys = pairs = blocks = 0
    for g in range(case["groups"]):
        common, used = prefix[g] // BLOCK * BLOCK, False
        for n in lens[first[g]:first[g + 1]]:
            if n:
                used = True
                keys += n - common
                blocks += -(-(n - common) // BLOCK)
                pairs += sum(n - T + t + 1 for t in range(T))
        keys += common if used else 0
        blocks += common // BLOCK if used else 0
    return {"bytes": 2 * keys * H * D + blocks * (8 * H + 4) + 2 * size * case["S"] * T * H * G * D, "flops": 4 * pairs * H * G * D}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    op, D = case["op"], case["dim"]
    st = prepare(case, seed)
    f64 = torch.float64
    if op in ("rope", "read"):
        lens, counts = _lengths(case["S"], case["longest"]), _counts(case)
        where = torch.cat([torch.arange(n - c, n, device="cuda") for n, c in zip(lens, counts)])
        if op == "read":
            of = torch.cat([torch.full((c,), s, device="cuda") for s, c in enumerate(counts)])
            blk = st["table"][of, where // BLOCK].long()
            k = st["k"][blk, :, where % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["k_scale"][blk, :, None].to(f64)
            v = st["v"][blk, :, :, where % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["v_scale"][blk, :, None].to(f64)
            return [k, v]
        rot = case["rot"]
        out = []
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + rot // 2)
        turn = torch.polar(torch.full((1,), st["factor"], dtype=f64, device="cuda"),
                           where.to(f64)[:, None] * st["inv_freq"].to(f64)[None])[:, None]
        for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
            y = x.to(f64)
            if w is not None:
                y = y * w.to(f64) / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6)
            z = torch.complex(y[..., a], y[..., b]) * turn
            y = y.clone()
            y[..., a], y[..., b] = z.real, z.imag
            out.append(y)
        return out
    S, T, H, G = case["S"], case["T"], case["heads"], case["group"]
    _, _, lens = _shape(case)
    if sum(lens) * T * H * G * D > 3e12:
        return None
    out = torch.zeros(S, T, H * G, D, dtype=f64, device="cuda")
    table = st["table"].long()
    for s in range(S):  # one sequence at a time, all of its blocks its own
        n = lens[s]
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        blk = table[s, j // BLOCK]
        late = j[None] > (n - T + torch.arange(T, device="cuda"))[:, None]
        for h in range(H):
            k = st["k"][blk, h, j % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["k_scale"][blk, h, None].to(f64)
            v = st["v"][blk, h, :, j % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["v_scale"][blk, h, None].to(f64)
            x = torch.einsum("tgd,nd->tgn", st["q"][s, :, h * G:(h + 1) * G].to(f64), k) / math.sqrt(D)
            x[late[:, None].expand_as(x)] = -math.inf
            out[s, :, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out
