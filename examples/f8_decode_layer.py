"""Attention half of a decoder layer in 8 bits, token by token, with libgemv's operators.

    python examples/f8_decode_layer.py [--steps N]

For each new token of a batch of sequences:

    gemv_f8_quantize   hidden state -> e4m3 with a scale per 128 channels
    gemv_f8            QKV projection (e4m3 weights, a scale per 128 x 128 block)
    gemv_kv8_append    the new keys and values into the 8-bit cache
    gemv_kv8_attention over the cache (grouped heads; a window and sinks if asked for)
    gemv_f8_quantize   attention output -> e4m3
    gemv_f8            output projection

One step is captured into a CUDA graph and replayed: lengths live on the device, so each
replay writes and reads one token further.  Weights, prompts and hidden states are random;
the printed error compares the last step with the same layer in 32 bits over the values
that the cache and the weights stand for.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import decode_linear_layers_gb300 as g  # noqa: E402

E4M3 = torch.float8_e4m3fn


def quantize_weights(w):
    """e4m3 weights and a scale for each block of 128 x 128."""
    M, K = w.shape
    gm, gk = -(-M // g.F8_GROUP), -(-K // g.F8_GROUP)
    p = torch.zeros(gm * g.F8_GROUP, gk * g.F8_GROUP, device=w.device)
    p[:M, :K] = w
    p = p.view(gm, g.F8_GROUP, gk, g.F8_GROUP)
    s = (p.abs().amax((1, 3)) / 448).clamp_min(2.0 ** -126)
    q = (p / s[:, None, :, None]).to(E4M3)
    return q.view(gm * g.F8_GROUP, gk * g.F8_GROUP)[:M, :K].contiguous(), s.contiguous()


def dequantized(q, s):
    M, K = q.shape
    return q.float() * s.repeat_interleave(g.F8_GROUP, 0)[:M].repeat_interleave(g.F8_GROUP, 1)[:, :K]


class Layer:
    """Weights, cache and buffers of a batch of S sequences of up to `longest` tokens."""

    def __init__(self, S, hidden, heads, group, dim, longest, window=0, sinks=0, seed=0):
        r = torch.Generator(device="cuda").manual_seed(seed)
        self.S, self.hidden, self.heads, self.q_heads, self.dim = S, hidden, heads, heads * group, dim
        self.window, self.sinks = window, sinks
        rows = (self.q_heads + 2 * heads) * dim
        self.w_qkv = quantize_weights(torch.randn(rows, hidden, generator=r, device="cuda") / math.sqrt(hidden))
        self.w_out = quantize_weights(torch.randn(hidden, self.q_heads * dim, generator=r, device="cuda") / math.sqrt(self.q_heads * dim))
        width = -(-longest // g.KV8_BLOCK)
        blocks = S * width
        self.k = torch.zeros(blocks, heads, g.KV8_BLOCK, dim, dtype=torch.uint8, device="cuda")
        self.v = torch.zeros(blocks, heads, dim, g.KV8_BLOCK, dtype=torch.uint8, device="cuda")
        self.ks, self.vs = torch.ones(blocks, heads, device="cuda"), torch.ones(blocks, heads, device="cuda")
        self.table = torch.randperm(blocks, generator=r, device="cuda").to(torch.int32).view(S, width)
        self.lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        self.x = torch.zeros(S, hidden, dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.empty(S, rows, dtype=torch.bfloat16, device="cuda")
        self.mixed = torch.empty(S, self.q_heads * dim, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(S, hidden, dtype=torch.bfloat16, device="cuda")

    def cache(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def linear(self, x, weights, y):
        """y = x W^T, x quantized on the way."""
        B, K = x.shape
        q = torch.empty(B, K, dtype=E4M3, device="cuda")
        s = torch.empty(B, -(-K // g.F8_GROUP), device="cuda")
        g.gemv_f8_quantize("bf16", x, q, s, K, B)
        g.gemv_f8(*weights, q, s, None, y, y.shape[1], K, B)

    def split(self, qkv):
        """Queries, keys and values: columns of the projection's output."""
        n, d = qkv.shape[0], self.dim
        a, b = self.q_heads * d, (self.q_heads + self.heads) * d
        return (qkv[:, :a].view(n, self.q_heads, d), qkv[:, a:b].view(n, self.heads, d), qkv[:, b:].view(n, self.heads, d))

    def prompt(self, x, counts):
        """The prompts' keys and values into the cache.  (This one layer can decode from them
        without their attention; a layer above it would need that for its own keys.)"""
        qkv = torch.empty(x.shape[0], self.qkv.shape[1], dtype=torch.bfloat16, device="cuda")
        self.linear(x, self.w_qkv, qkv)
        _, k, v = self.split(qkv)
        starts = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
        self.lens += starts[1:] - starts[:-1]
        g.gemv_kv8_append("bf16", *self.cache(), k, v, self.lens, starts, self.S, x.shape[0])

    def step(self):
        """One more token for each sequence, from self.x to self.y."""
        self.lens += 1
        self.linear(self.x, self.w_qkv, self.qkv)
        q, k, v = self.split(self.qkv)
        g.gemv_kv8_append("bf16", *self.cache(), k, v, self.lens, None, self.S, self.S)
        g.gemv_kv8_attention("bf16", *self.cache(), q, self.lens, self.mixed, None, self.S, 1, self.q_heads,
                             1 / math.sqrt(self.dim), window=self.window, sinks=self.sinks)
        self.linear(self.mixed, self.w_out, self.y)

    def plain(self):
        """The last step's output in 32 bits, from the projection's output on: attention over
        the values that the cache stands for, and the output projection."""
        q, _, _ = self.split(self.qkv)
        out = torch.zeros(self.S, self.q_heads, self.dim, device="cuda")
        for s, n in enumerate(self.lens.tolist()):
            j = torch.arange(n, device="cuda")
            if self.window:
                j = j[(n - 1 - j < self.window) | (j < self.sinks)]
            blk = self.table[s, j // g.KV8_BLOCK].long()
            k = self.k.view(E4M3).float()[blk, :, j % g.KV8_BLOCK] * self.ks[blk][..., None]
            v = self.v.view(E4M3).float()[blk, :, :, j % g.KV8_BLOCK] * self.vs[blk][..., None]
            group = self.q_heads // self.heads
            k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
            w = torch.softmax(torch.einsum("hd,nhd->hn", q[s].float(), k) / math.sqrt(self.dim), -1)
            out[s] = torch.einsum("hn,nhd->hd", w, v)
        return out.view(self.S, -1) @ dequantized(*self.w_out).t()


def run(steps=8, S=16, hidden=4096, heads=8, group=4, dim=128, prompt=1000, window=0, sinks=0, seed=0):
    """(relative error of the last step's output, us a step); see the module's text."""
    r = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Layer(S, hidden, heads, group, dim, prompt + steps + 4, window, sinks, seed)
    counts = [max(1, prompt * (i + 1) // S) for i in range(S)]
    layer.prompt(torch.randn(sum(counts), hidden, generator=r, device="cuda").to(torch.bfloat16), counts)
    hiddens = torch.randn(steps + 1, S, hidden, generator=r, device="cuda").to(torch.bfloat16)
    layer.x.copy_(hiddens[0])
    layer.step()                        # (the first call of each kernel is not captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for i in range(steps):
        layer.x.copy_(hiddens[i + 1])
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    want = layer.plain()
    error = float((layer.y.float() - want).norm() / want.norm())
    return error, begin.elapsed_time(end) / steps * 1e3


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    run(2)
    error, us = run(a.steps, window=a.window, sinks=a.sinks)
    print(f"16 sequences of up to 1000 tokens, hidden 4096, 32 query and 8 key heads of 128: {us:.1f} us a step, "
          f"relative error {error:.4f} (the quantized attention output among it)")
