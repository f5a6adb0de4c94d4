"""The block-scaled 8-bit floating point product (gemv_f8) and the quantiser of its
vectors (gemv_f8_quantize), against plain implementations in 64 bits.

Tolerances.  The quantiser: scales are one fp32 division, within 2^-23 of the exact
quotient; a value is x times a rounded reciprocal, so within 2^-22 of the exact x / s
before its rounding to e4m3, whose spacing at v is max(2^-9, 2^(floor(log2 |v|) - 3)):
the stored value lies within half that spacing (and 2^-22 |v|) of x / s.
The product: the sums are fp32 (the groups' in the tensor cores, the sum over groups in
registers): 1e-5 of sum |terms| as for the library's fp32 products, plus the output
type's unit roundoff of |y|.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _no_stall():
    g.test_stall(False)
    yield
    g.test_stall(False)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ the quantiser
def quantize(x, name):
    B, K = x.shape
    q = torch.full((B, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((B, -(-K // 128)), -1.0, device="cuda")
    g.gemv_f8_quantize(name, x, q, s, K, B)
    return q.view(E4M3), s


def check_quantized(x, q, s):
    B, K = x.shape
    G = -(-K // 128)
    xd = x.double()
    p = torch.nn.functional.pad(torch.where(torch.isfinite(xd), xd.abs(), torch.zeros_like(xd)), (0, G * 128 - K))
    ref = (p.view(B, G, 128).amax(2) / 448).clamp_min(2.0 ** -126)
    assert bool(((s.double() - ref).abs() <= 2.0 ** -23 * ref).all())
    v = xd / s.double().repeat_interleave(128, 1)[:, :K]
    got = q.float().double()
    assert torch.equal(torch.isnan(got), torch.isnan(v))
    ok = ~torch.isnan(v)
    v, got = v[ok].clamp(-448, 448), got[ok]
    # e4m3's spacing at |v|: 2^(floor(log2 |v|) - 3), 2^-9 below its smallest normal 2^-6
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    assert bool(((got - v).abs() <= 0.5 * step + 2.0 ** -22 * v.abs()).all())


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("B,K", [(1, 1), (1, 4096), (3, 127), (5, 128), (2, 129), (7, 264), (33, 1000), (4, 16384), (1025, 4096)])
def test_quantize(name, B, K):
    x = (torch.randn(B, K, generator=gen(B + K), device="cuda") * 5).to(TYPES[name])
    check_quantized(x, *quantize(x, name))


@pytest.mark.parametrize("name", TYPES)
def test_quantize_specials(name):
    x = torch.randn(6, 300, generator=gen(1), device="cuda")
    x[0] = 0
    x[1, 5], x[1, 200] = math.inf, -math.inf
    x[2, 7] = math.nan
    x[3] *= 1e-6      # fp16: subnormal
    x[4, :128] = math.inf
    x[5] = 448.0
    x = x.to(TYPES[name])
    q, s = quantize(x, name)
    check_quantized(x, q, s)
    f = q.float()
    assert f[1, 5] == 448 and f[1, 200] == -448 and torch.isnan(f[2, 7])
    assert s[0, 0] == 2.0 ** -126 and s[4, 0] == 2.0 ** -126 and bool((f[0] == 0).all())
    assert bool((f[5] == 448).all()) and bool((s[5] == 1).all())


@pytest.mark.parametrize("name", TYPES)
def test_quantize_unaligned(name):
    # rows that start anywhere: element loads; the bytes around q stay
    base = torch.randn(4 * 200 + 1, generator=gen(2), device="cuda").to(TYPES[name])
    x = base[1:].view(4, 200)
    buf = torch.full((4 * 200 + 34,), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.empty(4, 2, device="cuda")
    g.gemv_f8_quantize(name, x, buf[17:17 + 800], s, 200, 4)
    check_quantized(x, buf[17:17 + 800].view(4, 200).clone().view(E4M3), s)
    assert bool((buf[:17] == 0xEE).all()) and bool((buf[817:] == 0xEE).all())
    # and the same values as from aligned rows
    q2, s2 = quantize(x.contiguous().clone(), name)
    assert torch.equal(s, s2) and torch.equal(buf[17:817].view(4, 200), q2.view(torch.uint8))


# ------------------------------------------------------------------ the product
def operands(M, K, B, seed, scales=(0.25, 4.0)):
    r = gen(seed)
    G = -(-K // 128)
    A = torch.randn(M, K, generator=r, device="cuda").to(E4M3)
    x = (torch.randn(B, K, generator=r, device="cuda") * 20).to(E4M3)
    lo, hi = scales
    sa = lo * (hi / lo) ** torch.rand(-(-M // 128), G, generator=r, device="cuda")
    sx = lo * (hi / lo) ** torch.rand(B, G, generator=r, device="cuda")
    return A, sa, x, sx


def reference(A, sa, x, sx, bias):
    """(y, sum |terms|) in 64 bits."""
    M, K = A.shape
    a = A.float().double() * sa.double().repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    v = x.float().double() * sx.double().repeat_interleave(128, 1)[:, :K]
    y, mag = v @ a.t(), v.abs() @ a.abs().t()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    return y, mag


def product(A, sa, x, sx, bias, name, stream=None):
    (M, K), B = A.shape, x.shape[0]
    y = torch.full((B, M), float("nan"), dtype=TYPES[name], device="cuda")
    g.gemv_f8(A, sa, x, sx, bias, y, M, K, B, y_dtype=name, stream=stream)
    return y


def check_product(y, ref, mag, name):
    err = (y.double() - ref).abs()
    bound = 1e-5 * mag + ROUND[name] * ref.abs() + (2.0 ** -25 if name == "f16" else 0)
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())


# vectors: each form's ends; rows and columns: below, at and past whole tiles and blocks
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("B", [1, 2, 16, 17, 32, 33, 64, 65, 128, 129, 256, 385])
def test_product(name, B):
    for i, (M, K) in enumerate(((1, 16), (128, 128), (129, 144), (255, 256), (300, 1040), (1000, 528))):
        A, sa, x, sx = operands(M, K, B, seed=100 * B + i)
        bias = torch.randn(M, generator=gen(i), device="cuda").to(TYPES[name]) if i % 2 else None
        y = product(A, sa, x, sx, bias, name)
        check_product(y, *reference(A, sa, x, sx, bias), name)
        y2 = product(A, sa, x, sx, bias, name)
        assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8)), "two identical calls differ"
    assert g.device_status() == (0, 0)


# more tiles than SMs (whole tiles and shared ones), and one tile whose columns all share
@pytest.mark.parametrize("M,K,B", [(20000, 384, 4), (40000, 256, 40), (128, 16384, 1), (7000, 272, 1000), (256, 8192, 130),
                                   (39168, 128, 16),
                                   # pairs of SMs: one tile of 256 vectors, several, ragged ends
                                   (40000, 272, 200), (39937, 144, 300), (10250, 400, 1100), (4100, 16, 2600)])
def test_product_many_tiles(M, K, B):
    A, sa, x, sx = operands(M, K, B, seed=M)
    y = product(A, sa, x, sx, None, "bf16")
    check_product(y, *reference(A, sa, x, sx, None), "bf16")


# clusters for all tiles, and for those left over after rounds of whole ones
@pytest.mark.parametrize("M,K,B,name", [(301, 4112, 1, "bf16"), (300, 4096, 17, "f16"), (131, 8192, 40, "f32"), (700, 6160, 65, "bf16"),
                                        (1001, 8192, 129, "f32"), (3000, 8192, 200, "f16"), (516, 14336, 128, "f32"),
                                        (20353, 4096, 2, "bf16"), (24001, 3600, 40, "f32"), (21000, 7168, 30, "f16"),
                                        (42000, 2064, 1, "f32"), (24000, 3600, 100, "bf16"), (14301, 4096, 300, "f16"),
                                        (10004, 8192, 257, "f32"), (4097, 14336, 700, "bf16")])
def test_product_clusters(M, K, B, name):
    A, sa, x, sx = operands(M, K, B, seed=13)
    bias = torch.randn(M, generator=gen(14), device="cuda").to(TYPES[name])
    y = product(A, sa, x, sx, bias, name)
    check_product(y, *reference(A, sa, x, sx, bias), name)
    assert torch.equal(y, product(A, sa, x, sx, bias, name))
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("M,K,B", [(301, 4112, 1), (700, 6160, 65), (20353, 4096, 2), (14301, 4096, 300)])
def test_bounded_wait_in_clusters(M, K, B):
    A, sa, x, sx = operands(M, K, B, seed=15)
    torch.cuda.synchronize()
    g.test_stall(True, 50_000_000)
    product(A, sa, x, sx, None, "bf16")
    status, bits = g.device_status()
    assert status == g.ERR_DEVICE_TIMEOUT and bits & 16
    g.test_stall(False)
    check_product(product(A, sa, x, sx, None, "bf16"), *reference(A, sa, x, sx, None), "bf16")
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("B", [3, 200])
def test_product_scales_apart(B):
    # neighbouring groups whose scales differ by many orders: each group's own counts
    A, sa, x, sx = operands(200, 640, B, seed=5, scales=(1e-12, 1e12))
    y = product(A, sa, x, sx, None, "f32")
    check_product(y, *reference(A, sa, x, sx, None), "f32")


# (every form: up to 16, 32, 64 vectors, 128 and 256 weight rows a tile, pairs of SMs)
@pytest.mark.parametrize("M,K,B", [(300, 656, 1), (300, 656, 20), (300, 656, 50), (300, 656, 100), (12000, 272, 300), (40000, 272, 200)])
def test_product_scales_at_the_ends(M, K, B):
    """sa sx at the ends of what it may be, fp32's normal range (and 0), each scale far from 1."""
    # above: e4m3's subnormals, so that a group's sum is at most 128 x (7 x 2^-9)^2 < 2^-5
    r = gen(16)
    A, x = ((torch.randint(-7, 8, (n, K), generator=r, device="cuda") * 2.0 ** -9).to(E4M3) for n in (M, B))
    _, sa, _, sx = operands(M, K, B, seed=17, scales=(1.0, 2.0 ** 0.5))
    sa, sx = sa * 2.0 ** 66, sx * 2.0 ** 60.9   # 2^126.9 to 2^127.9
    x[B // 2], sx[B // 2] = 0, 2.0 ** 61
    y = product(A, sa, x, sx, None, "f32")
    check_product(y, *reference(A, sa, x, sx, None), "f32")
    assert bool((y[B // 2] == 0).all())
    # below; and a scale of 0
    A, sa, x, sx = operands(M, K, B, seed=18, scales=(1.0, 4.0))
    sa, sx = sa * 2.0 ** -86, sx * 2.0 ** -40   # 2^-126 to 2^-122
    sa[0, 0], sx[B // 2, 1] = 0, 0
    y = product(A, sa, x, sx, None, "f32")
    check_product(y, *reference(A, sa, x, sx, None), "f32")
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("B", [2, 150])
def test_product_nan_stays_in_its_row(B):
    A, sa, x, sx = operands(300, 256, B, seed=6)
    A.view(torch.uint8)[17, 3] = 0x7F
    x.view(torch.uint8)[1, 200] = 0x7F
    y = product(A, sa, x, sx, None, "bf16")
    nan = torch.isnan(y)
    want = torch.zeros_like(nan)
    want[:, 17] = True
    want[1] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("B", [1, 20, 140])
def test_product_guard_bytes(B):
    M, K = 333, 272
    A, sa, x, sx = operands(M, K, B, seed=7)
    for name, pad in (("bf16", 3), ("f32", 5)):   # y anywhere, its rows unaligned
        buf = torch.full((B * M + 2 * pad,), 7.0, dtype=TYPES[name], device="cuda")
        g.gemv_f8(A, sa, x, sx, None, buf[pad:pad + B * M], M, K, B, y_dtype=name)
        check_product(buf[pad:pad + B * M].view(B, M), *reference(A, sa, x, sx, None), name)
        assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all())


def test_product_empty():
    bias = torch.randn(50, device="cuda").to(torch.bfloat16)
    y = torch.empty(3, 50, dtype=torch.bfloat16, device="cuda")
    g.gemv_f8(None, None, None, None, bias, y, 50, 0, 3)
    assert torch.equal(y, bias.expand(3, 50))
    g.gemv_f8(None, None, None, None, None, y, 50, 0, 3)
    assert bool((y == 0).all())
    g.gemv_f8(None, None, None, None, None, None, 0, 16, 3)
    g.gemv_f8(None, None, None, None, None, None, 5, 16, 0)
    g.gemv_f8_quantize("bf16", None, None, None, 0, 4)


def test_product_on_a_stream_and_in_a_graph():
    s = torch.cuda.Stream()
    for B in (2, 200):
        A, sa, x, sx = operands(500, 512, B, seed=B)
        want = product(A, sa, x, sx, None, "bf16")
        torch.cuda.synchronize()
        got = product(A, sa, x, sx, None, "bf16", stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        y = torch.zeros_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gemv_f8(A, sa, x, sx, None, y, 500, 512, B)
        for _ in range(2):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_quantized_product_end_to_end():
    # quantize, then multiply: the definition on the stored 8-bit values
    B, K, M = 9, 1000 * 16, 130
    x = torch.randn(B, K, generator=gen(3), device="cuda").to(torch.bfloat16)
    q, s = quantize(x, "bf16")
    A, sa, _, _ = operands(M, K, 1, seed=3)
    check_product(product(A, sa, q, s, None, "f32"), *reference(A, sa, q, s, None), "f32")


# (clusters of few tiles, whole tiles, tiles that CTAs share; a tile's columns and rows)
@pytest.mark.parametrize("M,K,B", [(300, 512, 1), (300, 512, 200), (20000, 256, 2), (12000, 4096, 3), (40000, 256, 200)])
def test_bounded_wait(M, K, B):
    A, sa, x, sx = operands(M, K, B, seed=8)
    torch.cuda.synchronize()
    g.test_stall(True, 50_000_000)
    product(A, sa, x, sx, None, "bf16")
    status, bits = g.device_status()
    assert status == g.ERR_DEVICE_TIMEOUT and bits & 16
    g.test_stall(False)
    y = product(A, sa, x, sx, None, "bf16")
    check_product(y, *reference(A, sa, x, sx, None), "bf16")
    assert g.device_status() == (0, 0)


@pytest.mark.parametrize("M,K,B", [(40000, 1040, 200), (39937, 256, 300), (40000, 128, 200)])
@pytest.mark.parametrize("cta", [0, 1])
def test_bounded_wait_in_pairs(M, K, B, cta):
    """One CTA of a pair has begun copies that the other has not: all that are in flight are
    waited for (no bit 32) before the pair leaves."""
    A, sa, x, sx = operands(M, K, B, seed=8)
    torch.cuda.synchronize()
    g.test_stall(2 + cta, 50_000_000)
    product(A, sa, x, sx, None, "bf16")
    assert g.device_status() == (g.ERR_DEVICE_TIMEOUT, 16)
    g.test_stall(False)
    y = product(A, sa, x, sx, None, "bf16")
    check_product(y, *reference(A, sa, x, sx, None), "bf16")
    assert g.device_status() == (0, 0)


def test_refusals_on_real_buffers():
    A, sa, x, sx = operands(64, 64, 2, seed=9)
    y = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")

    def refused(*a, **k):
        with pytest.raises(g.GemvError) as e:
            g.gemv_f8(*a, **k)
        assert e.value.status == g.ERR_INVALID_VALUE

    refused(A, sa, x, sx, None, y, 64, 63, 2)                       # columns: no whole 16 bytes
    refused(A.view(-1)[1:], sa, x, sx, None, y, 63, 64, 2)          # rows not 16-byte aligned
    refused(A, sa, x.view(-1)[8:], sx, None, y, 64, 64, 1)
    refused(A, sa, x, sx, None, A.view(torch.bfloat16), 64, 64, 2)  # y over A
    with pytest.raises(ValueError):
        g.gemv_f8(A, sa, x, sx, None, y, 65, 64, 2)
    with pytest.raises(ValueError):
        g.gemv_f8(A, sa, x, sx, None, y, 64, 64, 2, y_dtype="f32")
    with pytest.raises(ValueError):
        g.gemv_f8_quantize("f32", x, x, sx, 64, 2)
