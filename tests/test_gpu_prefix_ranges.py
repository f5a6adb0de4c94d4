"""gemv_kv8_prefix_attention at the ends of its ranges: logits far below zero, values of
the smallest scales.

Tolerances: those of tests/test_gpu_prefix.py.
"""
from __future__ import annotations

import math

import pytest
import torch

import decode_linear_layers_gb300 as g
from tests.test_gpu_kv8 import BLOCK, E4M3, ROUND, attend, attention_reference
from tests.test_gpu_prefix import Shared, call, check, queries, small_weights

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
