"""GPU: the 8-bit cache's operators over batches of more sequences than a warp and than a CTA has threads (384 in
the few-row kernel, 512 in the tiled one), many of them empty."""
import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from oracle import kv_fp8
from tests.attn_helpers import cu_of, f64
from tests.fp8_helpers import PagedFp8, assert_close, reference, rows, run

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H, HK, D, SCALE = 4, 2, 64, 0.125


def lengths(count, seed, longest):
    """Short lengths, a third of them zero, with empty runs at both ends and a few long ones."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, longest + 1, count) * (rng.random(count) > 0.33)
    n[:count // 10] = 0
    n[-(count // 20):] = 0
    n[rng.choice(count, 3, replace=False)] = [130, 1, 257]
    return [int(x) for x in n]


@pytest.mark.parametrize("count", [33, 384, 385, 512, 513, 1000])
@pytest.mark.parametrize("max_q", [1, 64], ids=["few rows", "tiles"])
def test_attention(count, max_q):
    kv = lengths(count, count, 9)
    q_lens = [min(n, 3) for n in kv]
    cache = PagedFp8(kv, 16, HK, D, 3)
    q, out, lse = run(cache, q_lens, H, D, BF16, max_q=max_q)
    assert eg.engram_check_errors() == 0
    at = 0
    for i, n in enumerate(q_lens):
        if n:
            s = slice(at, at + n)
            assert_close(out[s], lse[s], *reference(cache, i, q[s], SCALE), BF16, D, SCALE, max_q * 2)
        at += n


@pytest.mark.parametrize("count", [33, 513, 1000])
def test_append_and_read(count):
    kv = lengths(count, count, 9)
    new = [min(n, 4) for n in kv]
    cache = PagedFp8(kv, 16, HK, D, 3)
    k, v = (rows((sum(new), HK, D), s, BF16).cuda() for s in (1, 2))
    desc = eg.make_attn_desc(H, HK, D)
    paged = (cache.kv_len, cache.table, *cache.tensors)
    eg.engram_kv_append_fp8(desc, k, v, cu_of(new), *paged)
    ko, vo = (torch.empty((sum(kv), HK, D), dtype=BF16, device="cuda") for _ in range(2))
    eg.engram_kv_read_fp8(desc, cu_of(kv), *paged, ko, vo)
    assert eg.engram_check_errors() == 0
    ko, vo, at, seen = f64(ko), f64(vo), 0, 0
    for i, (n, m) in enumerate(zip(new, kv)):
        for got, old, x in ((ko, cache.keys[i], k), (vo, cache.values[i], v)):
            want = np.concatenate([old[:m - n], kv_fp8.values(*kv_fp8.quantise(f64(x[at:at + n])))]) if n else old
            np.testing.assert_array_equal(got[seen:seen + m], want)
        at += n
        seen += m


@pytest.mark.parametrize("max_q", [1, 64], ids=["few rows", "tiles"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_values_stay_with_their_items(max_q, dtype):
    # many items one after the other in a worker, every third of which has a NaN code at its end, in another column
    kv = [1 + 7 * i % 40 for i in range(2000)]
    cache = PagedFp8(kv, 16, HK, D, 3)
    q_lens = [min(n, 2) for n in kv]
    q, clean, lse = run(cache, q_lens, H, D, dtype, max_q=max_q)
    for i in range(0, 2000, 3):
        page, slot = cache.place(i, kv[i] - 1, 1)
        cache.v[page, slot, i % HK, i % D] = 0x7F
    for _ in range(5):
        _, out, got = run(cache, q_lens, H, D, dtype, max_q=max_q, q=q)
        assert eg.engram_check_errors() == 0
        want = f64(clean).copy()
        last = np.cumsum(q_lens) - 1
        for i in range(0, 2000, 3):     # only the last token sees its own position
            of = i % HK * (H // HK)
            want[last[i], of:of + H // HK, i % D] = np.nan
        np.testing.assert_array_equal(np.isnan(f64(out)), np.isnan(want))
        np.testing.assert_allclose(f64(out), want, rtol=2 ** -7, atol=1e-4)
        np.testing.assert_array_equal(f64(got), f64(lse))
