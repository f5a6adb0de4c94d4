"""The 8-bit operators of a decode layer, as measured cases.

Four operators of one path: the quantiser of activation vectors (``quantize``), the
product of 8-bit floating point matrices with a scale for each block of 128
(``matmul``), the append of new tokens to an 8-bit cache of keys and values with a
scale for each block of 64 tokens and head (``append``), and the attention of the
newest tokens over that cache, over all of it or over a sliding window and the first
tokens (``attention``).

``run`` computes them in their plain form with elementary torch operations, in 32 bits
and rounded once (``own`` false), or calls the library (``own`` true).  ``exact`` is
the definition in 64 bits.

8-bit values are e4m3 (torch.float8_e4m3fn).
"""
import math

import torch

own = False

GROUP = 128   # elements (of a vector), or rows and columns (of a matrix), per scale
BLOCK = 64    # tokens of the cache per block
F8_MAX = 448.0
F8_TINY = 2.0 ** -126   # the smallest scale
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode vector before the QKV projection: latency
        {"name": "quantize_token", "op": "quantize", "type": "bf16", "B": 1, "K": 4096},
        # a prompt's hidden activations before the down projection
        {"name": "quantize_prompt", "op": "quantize", "type": "bf16", "B": 8192, "K": 14336},
        # the QKV projection of one decode vector: latency and weight bytes
        {"name": "matmul_token", "op": "matmul", "type": "bf16", "M": 6144, "K": 4096, "B": 1},
        # the gate and up projection of a decode batch: weight bytes
        {"name": "matmul_batch16", "op": "matmul", "type": "bf16", "M": 28672, "K": 4096, "B": 16},
        # odd rows and vectors, a last block of 16 columns, fp32 results (logits)
        {"name": "matmul_ragged", "op": "matmul", "type": "f32", "M": 10001, "K": 2064, "B": 77},
        # the down projection of a prompt: arithmetic
        {"name": "matmul_prompt", "op": "matmul", "type": "bf16", "M": 4096, "K": 14336, "B": 8192},
        # one new token for each sequence of a decode batch
        {"name": "append_token", "op": "append", "type": "bf16", "S": 64, "T": 1, "heads": 8, "dim": 128,
         "longest": 8192, "ragged": False},
        # prompts of different lengths written at once
        {"name": "append_prompt", "op": "append", "type": "f16", "S": 5, "T": 4096, "heads": 8, "dim": 128,
         "longest": 9000, "ragged": True},
        # a short conversation: latency
        {"name": "attention_short", "op": "attention", "type": "bf16", "S": 1, "T": 1, "heads": 8, "group": 4,
         "dim": 128, "longest": 100, "window": 0, "sinks": 0},
        # a decode batch of sequences of very different lengths
        {"name": "attention_batch", "op": "attention", "type": "bf16", "S": 64, "T": 1, "heads": 8, "group": 4,
         "dim": 128, "longest": 8192, "window": 0, "sinks": 0},
        # one sequence with a long cache
        {"name": "attention_long", "op": "attention", "type": "f16", "S": 1, "T": 1, "heads": 8, "group": 8,
         "dim": 128, "longest": 131072, "window": 0, "sinks": 0},
        # four drafted tokens checked at once, sliding window with visible first tokens,
        # blocks between the two given back
        {"name": "attention_window", "op": "attention", "type": "bf16", "S": 24, "T": 4, "heads": 4, "group": 6,
         "dim": 64, "longest": 20000, "window": 4096, "sinks": 4},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "append", "attention", "attention"])
    if op == "quantize":
        K = _spread(rng, 1, 16384)
        return {"op": op, "type": rng.choice(["bf16", "f16", "f32"]), "B": _spread(rng, 1, min(8192, 58_000_000 // K)),
                "K": K}
    if op == "matmul":
        M, K = _spread(rng, 16, 32768), 16 * _spread(rng, 1, 1024)
        return {"op": op, "type": rng.choice(["bf16", "bf16", "f16", "f32"]), "M": M, "K": K,
                "B": _spread(rng, 1, max(1, min(8192, 400_000_000_000 // (M * K), 200_000_000 // M)))}
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 192, 256])
    if op == "append":
        S, longest = _spread(rng, 1, 96), _spread(rng, 1, 9000)
        # cost: the whole cache is an output
        longest = max(1, min(longest, 400_000_000 // (S * heads * dim * 2)))
        return {"op": op, "type": rng.choice(["bf16", "f16", "f32"]), "S": S,
                "T": min(longest, rng.choice([1, 1, 3, _spread(rng, 1, 4096)])),
                "heads": heads, "dim": dim, "longest": longest, "ragged": rng.random() < 0.5}
    S, group = _spread(rng, 1, 96), rng.choice([1, 2, 3, 4, 6, 8, 16])
    longest = max(1, min(_spread(rng, 1, 131072), 134_000_000 // (S * heads * dim)))
    window = rng.choice([0, 0, _spread(rng, 1, 8192)])
    return {"op": op, "type": rng.choice(["bf16", "f16"]), "S": S, "T": rng.choice([1, 1, 1, 2, 4, 8]),
            "heads": heads, "group": group, "dim": dim, "longest": longest, "window": window,
            "sinks": rng.choice([0, 4, 64, 100]) if window else 0}


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Tokens of each sequence, the new ones among them: spread over (0, longest], the
    first sequence the longest."""
    return [max(1, math.ceil(case["longest"] * (1.0 - (i * 0.6180339887) % 1.0))) for i in range(case["S"])]


def _counts(case):
    """New tokens of each sequence (append): T, or spread over [0, T] where ragged."""
    n = [case["T"] if not case["ragged"] else int(case["T"] * (1.0 - (i * 0.3819660113) % 1.0)) for i in range(case["S"])]
    return [min(a, b) for a, b in zip(n, _lengths(case))]


def _rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _activations(gen, B, K, dtype):
    """Vectors with a few strong channels, as hidden states have them."""
    x = _rand(gen, B, K)
    x *= 1.0 + 30.0 * (torch.rand(K, generator=gen, device="cuda") < 0.004)
    return x.to(dtype)


def _quantized(x, rows):
    """(8-bit values, scales) of a matrix in blocks of `rows` x GROUP."""
    M, K = x.shape
    gm, gk = -(-M // rows), -(-K // GROUP)
    p = torch.zeros(gm * rows, gk * GROUP, device=x.device)
    p[:M, :K] = x
    p = p.view(gm, rows, gk, GROUP)
    s = (p.abs().amax(dim=(1, 3)) / F8_MAX).clamp_min(F8_TINY)
    q = (p * (1.0 / s)[:, None, :, None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    return q.reshape(gm * rows, gk * GROUP)[:M, :K].contiguous(), s.contiguous()


def _cache(gen, case, lens, written):
    """A cache that holds `written` tokens of each sequence: keys blocks x heads x BLOCK x
    dim, values blocks x heads x dim x BLOCK, scales blocks x heads, and the table of each
    sequence's blocks, scattered over the pool.  What is not written holds any bytes."""
    S, H, D = case["S"], case["heads"], case["dim"]
    width = max(1, -(-max(lens) // BLOCK))
    need = [-(-n // BLOCK) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    at = 0
    place = torch.full((S, width), -1, dtype=torch.int64)
    for i, n in enumerate(need):
        place[i, :n] = torch.arange(at, at + n)
        at += n
    place = place.cuda()
    table = torch.where(place >= 0, order[place.clamp_min(0)], torch.full_like(order[:1], -1))
    k = torch.empty(pool, H, BLOCK, D, dtype=torch.uint8, device="cuda")
    v = torch.empty(pool, H, D, BLOCK, dtype=torch.uint8, device="cuda")
    ks, vs = torch.empty(pool, H, device="cuda"), torch.empty(pool, H, device="cuda")
    for lo in range(0, pool, 512):
        n = min(512, pool - lo)
        level = torch.exp(0.3 * _rand(gen, n, H, 1, 1))
        for buf, sc, shape, c in ((k, ks, (n, H, BLOCK, D), 1.5), (v, vs, (n, H, D, BLOCK), 0.7)):
            x = _rand(gen, *shape) * level * c
            s = _power(x.abs().amax(dim=(2, 3)))
            buf[lo:lo + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            sc[lo:lo + n] = s
    # the last block of each sequence: bytes past its tokens are what the block held before
    last = torch.tensor([max(0, w - 1) // BLOCK for w in written], device="cuda")
    rest = torch.tensor([w - (max(0, w - 1) // BLOCK) * BLOCK for w in written], device="cuda")
    pb = table[torch.arange(S, device="cuda"), last].long()
    stale = (torch.arange(BLOCK, device="cuda")[None] >= rest[:, None])
    junk = torch.randint(0, 256, (S, H, BLOCK, D), generator=gen, device="cuda").to(torch.uint8)
    k[pb] = torch.where(stale[:, None, :, None], junk, k[pb])
    v[pb] = torch.where(stale[:, None, None, :], junk.transpose(2, 3), v[pb])
    return k, v, ks, vs, table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dtype = case["op"], TYPES[case["type"]]
    st = dict(case)
    if op == "quantize":
        B, K = case["B"], case["K"]
        st["x"] = _activations(gen, B, K, dtype)
        st["q"] = torch.empty(B, K, dtype=torch.float8_e4m3fn, device="cuda")
        st["s"] = torch.empty(B, -(-K // GROUP), device="cuda")
    elif op == "matmul":
        M, K, B = case["M"], case["K"], case["B"]
        st["A"], st["a_scale"] = _quantized(_rand(gen, M, K) * (0.5 / math.sqrt(K)), GROUP)
        st["x8"], st["x_scale"] = _quantized(_activations(gen, B, K, torch.float32), 1)
        st["bias"] = (_rand(gen, M) * 0.1).to(dtype)
        st["y"] = torch.empty(B, M, dtype=dtype, device="cuda")
    else:
        S, H, D = case["S"], case["heads"], case["dim"]
        lens = _lengths(case)
        if op == "append":
            counts = _counts(case)
            cache = _cache(gen, case, lens, [a - b for a, b in zip(lens, counts)])
            N = sum(counts)
            # keys and values are columns of the fused projection's output
            st["qkv"] = _rand(gen, N, 3 * H * D).to(dtype)
            st["new_k"] = st["qkv"][:, H * D:2 * H * D].view(N, H, D) if N else st["qkv"].view(0, H, D)
            st["new_v"] = st["qkv"][:, 2 * H * D:].view(N, H, D) if N else st["qkv"].view(0, H, D)
            starts = [0]
            for n in counts:
                starts.append(starts[-1] + n)
            # a batch where all sequences get T tokens needs no starts
            even = all(n == case["T"] for n in counts)
            st["starts"] = None if even else torch.tensor(starts, dtype=torch.int32, device="cuda")
            st["N"] = N
        else:
            cache = _cache(gen, case, lens, lens)
            G, T = case["group"], case["T"]
            st["q"] = _rand(gen, S, T, H * G, D).to(dtype)
            st["out"] = torch.empty(S, T, H * G, D, dtype=dtype, device="cuda")
            if case["window"]:  # blocks that no query sees any more were given back
                b = torch.arange(cache[4].shape[1], device="cuda")[None]
                n = torch.tensor(lens, device="cuda")[:, None]
                gone = (b * BLOCK >= case["sinks"]) & ((b + 1) * BLOCK <= n - T + 1 - case["window"])
                cache = (*cache[:4], torch.where(gone, torch.full_like(cache[4], -1), cache[4]))
        st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"] = cache
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _power(amax):
    """The smallest power of two s with amax <= 448 s (at least the smallest scale)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp_min(-126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)))


def _finite_amax(x, dim):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=dim)


def _to8(x):
    return x.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _plain_quantize(st):
    x = st["x"].float()
    B, K = x.shape
    G = -(-K // GROUP)
    p = torch.nn.functional.pad(x, (0, G * GROUP - K)).view(B, G, GROUP)
    s = (_finite_amax(p, 2) / F8_MAX).clamp_min(F8_TINY)
    q = _to8(p * (1.0 / s)[:, :, None])
    return [q.view(B, G * GROUP)[:, :K].contiguous(), s]


def _plain_matmul(st):
    M, K = st["M"], st["K"]
    a = st["A"].float() * st["a_scale"].repeat_interleave(GROUP, 0)[:M].repeat_interleave(GROUP, 1)[:, :K]
    x = st["x8"].float() * st["x_scale"].repeat_interleave(GROUP, 1)[:, :K]
    return (x @ a.t() + st["bias"].float()).to(st["y"].dtype)


def _plain_append(st):
    S, H, D, N = st["S"], st["heads"], st["dim"], st["N"]
    lens = st["lens"].long()
    i = torch.arange(N, device="cuda")
    if st["starts"] is None:
        starts = torch.arange(S + 1, device="cuda") * st["T"]
    else:
        starts = st["starts"].long()
    seq = torch.searchsorted(starts, i, right=True) - 1
    before = lens - (starts[1:] - starts[:-1])          # tokens held before
    pos = before[seq] + i - starts[seq]
    blk = st["table"][seq, pos // BLOCK].long()
    slot = pos % BLOCK
    # each sequence's open block (held tokens and new ones), if it has one
    some = (before % BLOCK > 0) & (starts[1:] > starts[:-1])
    first = st["table"].gather(1, (before // BLOCK).clamp_max(st["table"].shape[1] - 1)[:, None])[:, 0].long()
    held = torch.arange(BLOCK, device="cuda")[None] < (before % BLOCK)[:, None]
    held = held & some[:, None]

    def written(new, buf, sc, rows):  # rows: one per token (keys); else one per channel (values)
        new = new.float()
        amax = torch.zeros_like(sc).scatter_reduce(0, blk[:, None].expand(N, H), _finite_amax(new, 2), "amax")
        scale = sc.clone()
        scale[blk] = _power(amax)[blk]
        open_ = first[some]
        scale[open_] = torch.maximum(scale[open_], sc[open_])
        mask = held[some][:, None, :, None] if rows else held[some][:, None, None, :]
        old = buf[open_]
        moved = old.view(torch.float8_e4m3fn).float() * (sc[open_] / scale[open_])[:, :, None, None]
        buf[open_] = torch.where(mask, _to8(moved).view(torch.uint8), old)
        q = _to8(new / scale[blk][:, :, None]).view(torch.uint8)
        if rows:
            buf[blk, :, slot] = q
        else:
            buf[blk, :, :, slot] = q
        sc.copy_(scale)
        return [buf.view(torch.float8_e4m3fn), sc]

    return written(st["new_k"], st["k"], st["k_scale"], True) + written(st["new_v"], st["v"], st["v_scale"], False)


def _visible(st, n_keys):
    """S x T x keys: whether query t of a sequence sees the key at a position."""
    T, lens = st["T"], st["lens"].long()
    j = torch.arange(n_keys, device="cuda")[None, None]
    i = lens[:, None, None] - T + torch.arange(T, device="cuda")[None, :, None]
    see = j <= i
    if st["window"]:
        see = see & ((i - j < st["window"]) | (j < st["sinks"]))
    return see


def _gathered(st):
    """Keys (S x H x tokens x D) and values (S x H x D x tokens) in 32 bits."""
    S, H, D = st["S"], st["heads"], st["dim"]
    tab = st["table"].long().clamp_min(0)
    W = tab.shape[1]
    k = st["k"][tab].view(torch.float8_e4m3fn).float() * st["k_scale"][tab][..., None, None]
    v = st["v"][tab].view(torch.float8_e4m3fn).float() * st["v_scale"][tab][..., None, None]
    return (k.permute(0, 2, 1, 3, 4).reshape(S, H, W * BLOCK, D),
            v.permute(0, 2, 3, 1, 4).reshape(S, H, D, W * BLOCK))


def _plain_attention(st):
    S, T, H, G, D = st["S"], st["T"], st["heads"], st["group"], st["dim"]
    k, v = _gathered(st)
    see = _visible(st, k.shape[2])
    some = see.any(1)                                    # a key that no query sees is never read
    k = torch.where(some[:, None, :, None], k, torch.zeros_like(k[:1, :1, :1, :1]))
    v = torch.where(some[:, None, None, :], v, torch.zeros_like(v[:1, :1, :1, :1]))
    q = st["q"].float().view(S, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, T * G, D)
    s = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    s = s.view(S, H, T, G, -1).masked_fill(~see[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(S, H, T * G, -1) @ v.transpose(2, 3)).view(S, H, T, G, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(S, T, H * G, D).to(st["out"].dtype)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if not own:
        return {"quantize": _plain_quantize, "matmul": _plain_matmul, "append": _plain_append,
                "attention": _plain_attention}[op](st)
    import decode_linear_layers_gb300 as g
    if op == "quantize":
        g.gemv_f8_quantize(st["type"], st["x"], st["q"], st["s"], st["K"], st["B"])
        return [st["q"], st["s"]]
    if op == "matmul":
        g.gemv_f8(st["A"], st["a_scale"], st["x8"], st["x_scale"], st["bias"], st["y"], st["M"], st["K"], st["B"],
                  y_dtype=st["type"])
        return st["y"]
    cache = st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"]
    if op == "append":
        g.gemv_kv8_append(st["type"], *cache, st["new_k"], st["new_v"], st["lens"], st["starts"], st["S"], st["N"])
        return [st["k"].view(torch.float8_e4m3fn), st["k_scale"], st["v"].view(torch.float8_e4m3fn), st["v_scale"]]
    g.gemv_kv8_attention(st["type"], *cache, st["q"], st["lens"], st["out"], None, st["S"], st["T"],
                         st["heads"] * st["group"], 1.0 / math.sqrt(st["dim"]), window=st["window"], sinks=st["sinks"])
    return st["out"]


# ------------------------------------------------------------------ bytes and operations
def work(case):
    op, size = case["op"], {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    if op == "quantize":
        n = case["B"] * case["K"]
        return {"bytes": n * (size + 1) + 4 * case["B"] * -(-case["K"] // GROUP), "flops": 3 * n}
    if op == "matmul":
        M, K, B = case["M"], case["K"], case["B"]
        gk = -(-K // GROUP)
        return {"bytes": M * K + B * K + 4 * gk * (-(-M // GROUP) + B) + size * (M * B + M), "flops": 2 * M * K * B}
    S, H, D = case["S"], case["heads"], case["dim"]
    lens = _lengths(case)
    if op == "append":
        n = sum(_counts(case))
        # new tokens read and written, their blocks' scales and table entries
        blocks = sum(-(-a // BLOCK) - (a - b) // BLOCK for a, b in zip(lens, _counts(case)) if b)
        return {"bytes": 2 * n * H * D * (size + 1) + blocks * (8 * H + 4), "flops": 4 * n * H * D}
    T, G = case["T"], case["group"]
    keys = pairs = blocks = 0
    for n in lens:
        lo = max(0, n - T + 1 - case["window"]) if case["window"] else 0
        sinks = min(case["sinks"], lo, n)
        seen = max(0, n - lo) + sinks
        keys += seen
        blocks += -(-seen // BLOCK)
        for t in range(T):
            i = n - T + t
            a = max(0, i + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, i + 1 - a) + min(case["sinks"], a, max(0, i + 1))
    return {"bytes": 2 * keys * H * D + blocks * (8 * H + 4) + 2 * size * S * T * H * G * D, "flops": 4 * pairs * H * G * D}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    f64 = torch.float64
    if op == "quantize":
        x = st["x"].to(f64)
        K, B = case["K"], case["B"]
        s = torch.stack([x[:, g:g + GROUP].abs().amax(1) / F8_MAX for g in range(0, K, GROUP)], 1).clamp_min(F8_TINY)
        return [x / s[:, torch.arange(K, device="cuda") // GROUP], s]
    if op == "matmul":
        M, K, B = case["M"], case["K"], case["B"]
        y = st["bias"].to(f64).expand(B, M).clone()
        rows = torch.arange(M, device="cuda") // GROUP
        for g in range(-(-K // GROUP)):  # block by block of the columns: y += s_a s_x (A x)
            c = slice(g * GROUP, min(K, (g + 1) * GROUP))
            part = st["x8"][:, c].to(f64) @ st["A"][:, c].to(f64).t()
            part *= st["x_scale"][:, g, None].to(f64)
            part *= st["a_scale"][rows, g].to(f64)
            y += part
            del part
        return y
    if op == "append":  # the scales; the 8-bit values are held to the plain form's
        ends = [0]
        for n in _counts(case):
            ends.append(ends[-1] + n)
        table = st["table"].tolist()
        scales = []
        for new, sc in ((st["new_k"], st["k_scale"]), (st["new_v"], st["v_scale"])):
            new, sc = new.to(f64).abs(), sc.to(f64)
            for s, (n, c) in enumerate(zip(_lengths(case), _counts(case))):
                for b in range((n - c) // BLOCK, -(-n // BLOCK) if c else 0):
                    lo, hi = max(n - c, b * BLOCK), min(n, (b + 1) * BLOCK)
                    at = ends[s] + lo - (n - c)
                    need = 2.0 ** torch.ceil(torch.log2(new[at:at + hi - lo].amax((0, 2)) / F8_MAX))
                    pb = table[s][b]
                    sc[pb] = torch.maximum(need, sc[pb]) if lo % BLOCK else need
            scales.append(sc)
        return [None, scales[0], None, scales[1]]
    S, T, H, G, D = case["S"], case["T"], case["heads"], case["group"], case["dim"]
    lens = _lengths(case)
    out = torch.zeros(S, T, H * G, D, dtype=f64, device="cuda")
    table = st["table"].tolist()
    for s in range(S):  # one sequence at a time: its visible tokens, a softmax over them
        n = lens[s]
        for t in range(T):
            i = n - T + t
            if i < 0:
                continue
            j = torch.arange(i + 1, device="cuda")
            if case["window"]:
                j = j[(j > i - case["window"]) | (j < case["sinks"])]
            blk = torch.tensor(table[s], device="cuda")[j // BLOCK].long()
            for h in range(H):
                k = st["k"][blk, h, j % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["k_scale"][blk, h, None].to(f64)
                v = st["v"][blk, h, :, j % BLOCK].view(torch.float8_e4m3fn).to(f64) * st["v_scale"][blk, h, None].to(f64)
                w = torch.softmax(st["q"][s, t, h * G:(h + 1) * G].to(f64) @ k.t() / math.sqrt(D), -1)
                out[s, t, h * G:(h + 1) * G] = w @ v
    return out
