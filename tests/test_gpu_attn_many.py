"""GPU: batches of more sequences than a warp and than a CTA has threads (288 in the few-row kernel,
384 in the tiled one), many of them empty, against the float64 oracle: how a worker finds its range."""
import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from oracle.attention import attend
from tests.attn_helpers import Paged, assert_attn_close, cu_of, f64, randn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
COUNTS = [33, 288, 289, 384, 385, 1000]
H, HK, D = 4, 2, 64
SCALE = 0.125


def lengths(count, seed, longest):
    """Short lengths, a third of them zero, with empty runs at both ends and a few long ones."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, longest + 1, count) * (rng.random(count) > 0.33)
    n[:count // 10] = 0
    n[-(count // 20):] = 0
    n[rng.choice(count, 3, replace=False)] = [130, 1, 257]
    return [int(x) for x in n]


def check(out, lse, q, keys, values, lens):
    out, lse, q = out.cpu(), lse.cpu(), f64(q)
    at = 0
    for i, n in enumerate(lens):
        if n:
            ref = attend(q[at:at + n], f64(keys[i]), f64(values[i]), SCALE)
            assert_attn_close(out[at:at + n], lse[at:at + n], ref, BF16, D, SCALE)
        at += n


@pytest.mark.parametrize("count", COUNTS)
def test_prompts(count):
    lens = lengths(count, count, 5)
    total = sum(lens)
    q, k, v = (randn((total, h, D), s, BF16) for h, s in ((H, 1), (HK, 2), (HK, 3)))
    out, lse = torch.full_like(q, float("nan")), torch.full((total, H), 7.0, device="cuda")
    eg.engram_attn_prompt(eg.make_attn_desc(H, HK, D), q, k, v, cu_of(lens), out, lse_out=lse)
    assert eg.engram_check_errors() == 0
    check(out, lse, q, torch.split(k.cpu(), lens), torch.split(v.cpu(), lens), lens)


@pytest.mark.parametrize("max_q", [1, 64], ids=["few rows", "tiles"])
@pytest.mark.parametrize("count", COUNTS)
def test_chunks_over_caches(count, max_q):
    q_lens = lengths(count, count + 1, 2)
    kv_lens = [n + m for n, m in zip(q_lens, lengths(count, count + 2, 40))]
    cache = Paged(kv_lens, 16, HK, D, BF16, count)
    q = randn((sum(q_lens), H, D), 4, BF16)
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], 7.0, device="cuda")
    eg.engram_attn_paged(eg.make_attn_desc(H, HK, D), q, cu_of(q_lens), cache.kv_len, cache.table, cache.k,
                         cache.v, out, max_q, lse_out=lse)
    assert eg.engram_check_errors() == 0
    check(out, lse, q, cache.keys, cache.values, q_lens)


@pytest.mark.parametrize("count", COUNTS)
def test_append(count):
    q_lens = lengths(count, count + 3, 3)
    kv_lens = [n + m for n, m in zip(q_lens, lengths(count, count + 4, 20))]
    cache = Paged(kv_lens, 8, HK, D, BF16, count)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    k, v = randn((sum(q_lens), HK, D), 5, BF16), randn((sum(q_lens), HK, D), 6, BF16)
    at = 0
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):
        if n:
            p = cache.place(i, m - n, n)
            want_k[p], want_v[p] = k[at:at + n], v[at:at + n]
        at += n
    eg.engram_kv_append(eg.make_attn_desc(HK, HK, D), k, v, cu_of(q_lens), cache.kv_len, cache.table, cache.k,
                        cache.v)
    assert eg.engram_check_errors() == 0
    bits = torch.int16      # slots that nobody owns hold NaN
    assert torch.equal(cache.k.view(bits), want_k.view(bits)) and torch.equal(cache.v.view(bits), want_v.view(bits))
