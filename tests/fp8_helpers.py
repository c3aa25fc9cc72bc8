"""Inputs and tolerances of the tests of the 8-bit cache."""
from __future__ import annotations

import math

import numpy as np
import torch

import deepseek_v4_engram_gb300 as eg
from oracle import kv_fp8
from oracle.attention import attend
from oracle.numerics import e4m3_to_f64
from tests.attn_helpers import STEP, UNIT, cu_of, f64, randn


def rows(shape, seed, dtype=torch.bfloat16, spread=1.0):
    """Keys or values [..., D] whose sizes differ from row to row (by powers of two)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    return (x * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g))).to(dtype)


class PagedFp8:
    """A paged 8-bit cache whose pages are shuffled. Slots that no position owns hold NaN codes and NaN
    scales, page table entries past a sequence's end (`columns` more than the longest has) pages that do
    not exist."""

    def __init__(self, kv_lens, page, kv_heads, head_dim, seed, layout="nhd", spare=3, spread=1.0,
                 dtype=torch.bfloat16, device="cuda", columns=2):
        need = [-(-max(n, 0) // page) for n in kv_lens]
        pages, width = sum(need) + spare, max(need + [1]) + columns
        kw = dict(dtype=torch.uint8, device=device)
        if layout == "pool":        # a page's codes and scales one after the other, in one buffer
            part = page * kv_heads * head_dim
            row = 2 * part + 2 * kv_heads * page
            pool = torch.full((pages, row + 16 * 5), 255, **kw)
            self.k, self.v = (pool[:, i * part:(i + 1) * part].view(pages, page, kv_heads, head_dim) for i in range(2))
            self.k_scale, self.v_scale = (
                pool[:, 2 * part + i * kv_heads * page:2 * part + (i + 1) * kv_heads * page].view(pages, kv_heads, page)
                for i in range(2))
        else:
            shape = (pages, kv_heads, page, head_dim) if layout == "hnd" else (pages, page, kv_heads, head_dim)
            self.k, self.v = torch.full(shape, 0x7F, **kw), torch.full(shape, 0xFF, **kw)
            if layout == "hnd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
            self.k_scale, self.v_scale = (torch.full((pages, kv_heads, page), 255, **kw) for _ in range(2))
        order = np.random.default_rng(seed).permutation(pages)
        table = np.full((len(kv_lens), width), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.host_table, self.page = table, page
        self.table = torch.from_numpy(table).to(device)
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device=device)
        self.keys, self.values, self.codes, self.exponents = [], [], [], []
        for i, n in enumerate(kv_lens):
            kc, ks = kv_fp8.quantise(f64(rows((max(n, 0), kv_heads, head_dim), seed * 100 + 2 * i, dtype, spread)))
            vc, vs = kv_fp8.quantise(f64(rows((max(n, 0), kv_heads, head_dim), seed * 100 + 2 * i + 1, dtype, spread)))
            self.keys.append(kv_fp8.values(kc, ks))
            self.values.append(kv_fp8.values(vc, vs))
            self.codes.append(e4m3_to_f64(vc))
            self.exponents.append(vs.astype(np.int64) - 127)
            self.write(i, 0, kc, ks, vc, vs)

    def place(self, i, start, count):
        pos = np.arange(start, start + count)
        dev = self.k.device
        return (torch.from_numpy(self.host_table[i][pos // self.page].astype(np.int64)).to(dev),
                torch.from_numpy(pos % self.page).to(dev))

    def write(self, i, start, kc, ks, vc, vs):
        page, slot = self.place(i, start, kc.shape[0])
        for to, x in ((self.k, kc), (self.v, vc)):
            to[page, slot] = torch.from_numpy(x).to(to.device)
        for to, x in ((self.k_scale, ks), (self.v_scale, vs)):
            to[page, :, slot] = torch.from_numpy(x).to(to.device)

    @property
    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale


#: A call whose longest chunk has more rows (tokens x heads that share a key-value head) goes to the kernel
#: that computes on 16-bit tiles.
def few_rows(rows, head_dim):
    return rows <= (64 if head_dim <= 64 else 48)


def tolerance(ref, extra, dtype, head_dim, scale, rows):
    """How far out and lse may be from the exact ones (ref = attend(...) over the cache's values), for a call of
    `rows` rows.

    Few rows: codes and queries enter the products exactly, but for what of a query row lies 2^-39 below its
    largest element (`small`: what it adds to a score). The scores are f32 sums of head_dim products: off by at most
    e = (head_dim + 6) 2^-24 * scale sum_d |q_d k_d| + small, the products with the scales and the base of the
    logarithm included, so each probability is off by a factor of 1 +- (e + 2^-21). It is rounded to f16 times its
    value's scale: by 2^-11 relative, or by half of f16's smallest step, which is at most 2^-31 of the largest
    such product of the row (`steps`: summed over the keys with their codes). The sum of the probabilities brings
    e + 2^-21 once more, its own additions and the output's accumulation less than 2^-16 for the lengths
    here. The result is rounded once.

    More rows: keys and values are 16-bit tiles of exactly the cache's values (those of these tests have one in
    dtype), and a probability is rounded to dtype by itself, as over a 16-bit cache: by half a unit in its last
    place, 2^-8 in bf16 and 2^-11 in f16, or by half the type's smallest step against a sum that is at least 1.
    All else as above.
    """
    out, lse, mass, dot, vsum = ref
    small, steps = extra
    u = UNIT[dtype]
    few = few_rows(rows, head_dim)
    e = (head_dim + 6) * 2.0 ** -24 * dot + small + 2.0 ** -21 * (1 + dot / 16)
    t = ((2.0 ** -11 if few else u) + 2 * e + 2.0 ** -16)[..., None] * mass + (steps if few else STEP[dtype] * vsum)
    return t + u * (np.abs(out) + t) + STEP[dtype], e + 2.0 ** -16 + 2.0 ** -22 * np.abs(dot)


def reference(cache, i, q, scale):
    """attend() of sequence i's chunk q over its keys, and what the tolerance needs besides."""
    k, v, codes = cache.keys[i], cache.values[i], cache.codes[i]
    q = f64(q)
    n, H, D = q.shape
    m, Hk, _ = k.shape
    ref = attend(q, k, v, scale)
    small, steps = np.zeros((n, H)), np.zeros((n, H, D))
    for t in range(n):
        seen = m - n + t + 1
        if seen <= 0:
            continue
        for h in range(H):
            c = h // (H // Hk)
            s = scale * (k[:seen, c] @ q[t, h])
            w = np.exp(s - ref[1][t, h])
            contribution = np.ldexp(w, cache.exponents[i][:seen, c])
            steps[t, h] = 2.0 ** -31 * contribution.max() * np.abs(codes[:seen, c]).sum(0)
            small[t, h] = 2.0 ** -39 * np.abs(q[t, h]).max() * scale * np.abs(k[:seen, c]).sum(1).max()
    return ref, (small, steps)


def assert_close(got, lse, ref, extra, dtype, head_dim, scale, rows):
    t_out, t_lse = tolerance(ref, extra, dtype, head_dim, scale, rows)
    g = f64(got)
    assert np.isfinite(g).all(), f"{(~np.isfinite(g)).sum()} outputs are not finite"
    bad = np.abs(g - ref[0]) > t_out
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off; first {np.argwhere(bad)[:4]}, "
                           f"worst {np.max(np.abs(g - ref[0]) / t_out):.3g} of the tolerance")
    if lse is not None:
        n = f64(lse)
        empty = np.isneginf(ref[1])
        assert (np.isneginf(n) == empty).all(), "lse is -inf exactly where a row sees nothing"
        d = np.abs(np.where(empty, 0.0, n) - np.where(empty, 0.0, ref[1]))
        assert (d <= t_lse).all(), f"lse off by {d.max():.3g}"


def run(cache, q_lens, heads, head_dim, dtype, seed=2, max_q=None, stream=None, workspace=None, q_scale=1.0, q=None,
        scale=None):
    kv_heads = cache.k.shape[2]
    if q is None:
        q = randn((sum(q_lens), heads, head_dim), seed, dtype, q_scale)
    desc = eg.make_attn_desc(heads, kv_heads, head_dim, dtype, scale)
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    eg.engram_attn_paged_fp8(desc, q, cu_of(q_lens), cache.kv_len, cache.table, *cache.tensors, out,
                             max(q_lens) if max_q is None else max_q, workspace=workspace, lse_out=lse, stream=stream)
    return q, out, lse


def check(q_lens, kv_lens, page, heads, kv_heads, head_dim, dtype, seed=2, layout="nhd", spread=1.0, columns=2, **kw):
    cache = PagedFp8(kv_lens, page, kv_heads, head_dim, seed, layout, spread=spread, columns=columns)
    q, out, lse = run(cache, q_lens, heads, head_dim, dtype, seed, **kw)
    assert eg.engram_check_errors() == 0
    scale, at = kw.get("scale") or 1 / math.sqrt(head_dim), 0
    max_q = kw.get("max_q")
    n_rows = max(max(q_lens) if max_q is None else max_q, 1) * (heads // kv_heads)
    for i, n in enumerate(q_lens):
        s = slice(at, at + n)
        assert_close(out[s], lse[s], *reference(cache, i, q[s], scale), dtype, head_dim, scale, n_rows)
        at += n
