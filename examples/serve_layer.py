"""The Engram block and an attention beside it, served together: a batch of prompts, then one or several
tokens per sequence and step.

    python examples/serve_layer.py [--eight-bits]

One length array serves both caches: engram_forward appends the tokens to its look-back cache and
advances cache_len, and that same array is the kv_len of engram_kv_append and engram_attn_paged, or of
engram_kv_append_fp8 and engram_attn_paged_fp8 where the attention's cache is kept in eight bits. Random
weights; the projections around the attention are plain matrix products.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import deepseek_v4_engram_gb300 as eg  # noqa: E402
import synth  # noqa: E402


def dev(a):
    if a.dtype.kind == "u" and a.dtype.itemsize > 1:     # torch has no wide unsigned types: same bits
        a = a.view("i%d" % a.dtype.itemsize)
    return torch.from_numpy(a).cuda()


class Layer:
    """The block's tables and weights, the attention's projection, and both caches of a batch."""

    def __init__(self, geom: synth.Geometry, heads: int, kv_heads: int, head_dim: int, batch: int,
                 capacity: int, page: int, seed: int = 1, eight_bits: bool = False):
        m = synth.make_model(geom, seed)
        t = m.tables
        self.geom, self.heads, self.kv_heads, self.head_dim = geom, heads, kv_heads, head_dim
        self.desc = eg.make_desc(geom.dim, geom.hc_mult, geom.n_heads, geom.max_ngram_size, geom.head_dim,
                                 t.num_embeddings, m.eps)
        self.tables = eg.DeviceTables(dev(t.token_map), t.pad_id, dev(t.multipliers), dev(t.primes),
                                      dev(t.offsets))
        self.weights = eg.DeviceWeights(dev(m.table), dev(m.scales), dev(m.wkv), dev(m.q), dev(m.k))
        self.attn = eg.make_attn_desc(heads, kv_heads, head_dim)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.wqkv = (torch.randn((geom.dim, (heads + 2 * kv_heads) * head_dim), generator=g, device="cuda")
                     * geom.dim ** -0.5).to(torch.bfloat16)
        # the block's look-back cache
        self.ids = torch.zeros((batch, capacity), dtype=torch.int32, device="cuda")
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.started = False    # whether the caches hold anything
        # pages of the attention's cache, dealt to the sequences in turn
        per_seq = -(-capacity // page)
        pages = batch * per_seq
        shape, kind = (pages, page, kv_heads, head_dim), torch.float8_e4m3fn if eight_bits else torch.bfloat16
        self.eight_bits = eight_bits
        self.cache = tuple(torch.empty(shape, dtype=kind, device="cuda") for _ in range(2))   # keys, values
        if eight_bits:      # and a scale for each of their rows, in the order in which heads read them
            self.cache += tuple(torch.empty((pages, kv_heads, page), dtype=torch.float8_e8m0fnu, device="cuda")
                                for _ in range(2))
        self.table = torch.arange(batch * per_seq, dtype=torch.int32, device="cuda").view(per_seq, batch)
        self.table = self.table.t().contiguous()
        self.scratch = torch.empty(eg.engram_attn_workspace_size(self.attn), dtype=torch.uint8, device="cuda")

    def step(self, x, tokens):
        """x bf16 [B, T, hc, dim] and the T new tokens of each sequence (a prompt first, then any number at
        a time): returns the block's streams [B, T, hc, dim] and the queries, keys, values and attention
        outputs [B * T, heads, head_dim]."""
        B, T = tokens.shape
        first, self.started = not self.started, True    # a prompt's keys are all in hand: the cache is only filled
        streams = torch.empty_like(x)
        work = torch.empty(max(eg.engram_forward_workspace_size(self.desc, B * T), 256), dtype=torch.uint8,
                           device="cuda")
        eg.engram_forward(self.desc, self.tables, self.weights, x, tokens, self.ids, self.length, None,
                          streams, work)
        qkv = (streams.float().mean(2).to(torch.bfloat16).view(B * T, -1) @ self.wqkv).view(
            B * T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        out = torch.empty((B * T, self.heads, self.head_dim), dtype=torch.bfloat16, device="cuda")
        cu = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
        paged = (cu, self.length, self.table, *self.cache)
        (eg.engram_kv_append_fp8 if self.eight_bits else eg.engram_kv_append)(self.attn, k, v, *paged)
        if first:
            eg.engram_attn_prompt(self.attn, q, k, v, cu, out, workspace=self.scratch)
        else:
            attend = eg.engram_attn_paged_fp8 if self.eight_bits else eg.engram_attn_paged
            attend(self.attn, q, *paged, out, T, workspace=self.scratch)
        return streams, q, k, v, out

    def cached(self, n: int):
        """The keys and values [B * n, kv_heads, head_dim] of each sequence's last n positions, as the 8-bit cache
        holds them."""
        B = self.length.numel()
        k, v = (torch.empty((B * n, self.kv_heads, self.head_dim), dtype=torch.bfloat16, device="cuda")
                for _ in range(2))
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        eg.engram_kv_read_fp8(self.attn, cu, self.length, self.table, *self.cache, k, v)
        return k, v


def serve(batch: int = 3, prompt: int = 40, steps: int = 4, heads: int = 8, kv_heads: int = 2,
          head_dim: int = 64, page: int = 16, seed: int = 1, eight_bits: bool = False):
    """A prompt and `steps` decoding steps; returns the layer and what each call of step() returned."""
    geom = synth.TINY
    layer = Layer(geom, heads, kv_heads, head_dim, batch, prompt + steps, page, seed, eight_bits)
    got = []
    for i, n in enumerate([prompt] + [1] * steps):
        b = synth.make_batch(geom, batch, n, seed + 10 + i)
        got.append(layer.step(dev(b.x).view(torch.bfloat16), dev(b.tokens)))
    bits = eg.engram_check_errors()
    if bits:
        raise RuntimeError(f"device error word {bits:#x}")
    return layer, got


if __name__ == "__main__":
    layer, got = serve(eight_bits="--eight-bits" in sys.argv[1:])
    print("lengths", layer.length.tolist())
    for i, (streams, q, k, v, out) in enumerate(got):
        print("prompt" if i == 0 else f"step {i}", "out", list(out.shape), "rms %.4f" % out.float().pow(2).mean().sqrt())
