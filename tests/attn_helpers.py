"""Inputs and tolerances of the attention tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle.attention import attend

#: Half a unit in the last place of a 16-bit type, relative, and half its smallest step.
UNIT = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def tolerance(ref, dtype, head_dim, scale):
    """How far out and lse may be from the exact ones (ref = attend(...)).

    u is the type's relative rounding. The scores are f32 sums of head_dim products: off by at most
    e = (head_dim + 4) 2^-24 * scale sum_d |q_d k_d|, the products with the scale and the base of
    the logarithm included, so each probability is off by a factor of 1 +- (e + 2^-21) (2^-21: the
    exponential itself and the subtraction of the maximum), and by u once it is rounded for the
    product with the values (at least half the type's smallest step, against a sum that is at least
    1). The sum of the probabilities brings the same e + 2^-21 once more, its own additions and the
    output's accumulation less than 2^-16 for the lengths here. The result is rounded once.
    """
    out, lse, mass, dot, vsum = ref
    u = UNIT[dtype]
    e = (head_dim + 4) * 2.0 ** -24 * dot + 2.0 ** -21 * (1 + dot / 16)
    t = (u + 2 * e + 2.0 ** -16)[..., None] * mass + STEP[dtype] * vsum
    return t + u * (np.abs(out) + t) + STEP[dtype], e + 2.0 ** -16 + 2.0 ** -22 * np.abs(dot)


def assert_attn_close(got, lse, ref, dtype, head_dim, scale):
    t_out, t_lse = tolerance(ref, dtype, head_dim, scale)
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


def randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Paged:
    """A paged cache whose pages are shuffled, with every slot that no position owns, and every
    page table entry past a sequence's end, set to something that must not be read in earnest."""

    def __init__(self, kv_lens, page, kv_heads, head_dim, dtype, seed, layout="nhd", spare=3):
        need = [-(-n // page) for n in kv_lens]
        pages, width = sum(need) + spare, max(need + [1]) + 2
        shape = {"nhd": (pages, page, kv_heads, head_dim),
                 "hnd": (pages, kv_heads, page, head_dim),
                 "pair": (pages, 2, page, kv_heads, head_dim)}[layout]
        nan = float("nan")
        if layout == "pair":
            both = torch.full(shape, nan, dtype=dtype, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k = torch.full(shape, nan, dtype=dtype, device="cuda")
            self.v = torch.full(shape, nan, dtype=dtype, device="cuda")
            if layout == "hnd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = np.random.default_rng(seed).permutation(pages)
        table = np.full((len(kv_lens), width), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.host_table, self.page = table, page
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        self.keys, self.values = [], []
        for i, n in enumerate(kv_lens):
            k = randn((n, kv_heads, head_dim), seed * 100 + 2 * i, dtype)
            v = randn((n, kv_heads, head_dim), seed * 100 + 2 * i + 1, dtype)
            self.keys.append(k)
            self.values.append(v)
            self.write(i, 0, k, v)

    def place(self, i, start, count):
        pos = np.arange(start, start + count)
        return (torch.from_numpy(self.host_table[i][pos // self.page].astype(np.int64)).cuda(),
                torch.from_numpy(pos % self.page).cuda())

    def write(self, i, start, k, v):
        page, slot = self.place(i, start, k.shape[0])
        self.k[page, slot] = k
        self.v[page, slot] = v


def reference(q, k, v, scale):
    return attend(f64(q), f64(k), f64(v), scale)
