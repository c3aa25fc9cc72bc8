"""GPU: an infinite value counts with the probability it has, wherever in its sequence it lies: as an
infinity while the probability is not zero, and as NaN (zero times infinity) where it has underflowed,
in the tiles that every row sees and in those at the end that only later rows see."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from tests.attn_helpers import Paged, cu_of, f64, randn

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
D, N = 64, 400


@pytest.mark.parametrize("where", [N - 1, 40], ids=["at the end", "in the middle"])
@pytest.mark.parametrize("dtype,below,want", [(BF16, 20, "inf"), (F16, 20, "inf"), (F16, 28, "inf"),
                                              (BF16, 300, "nan"), (F16, 300, "nan")])
@pytest.mark.parametrize("q_len", [1, 4, 100])
def test_infinite_value_of_small_weight(q_len, dtype, below, want, where):
    """The last row's weight of the key is 2^-below of its largest."""
    cache = Paged([N], 16, 1, D, dtype, 41)
    q = randn((q_len, 1, D), 42, dtype)
    last, scale = q[-1, 0].double(), 1 / math.sqrt(D)
    keys = cache.keys[0][:, 0].double()
    others = torch.cat([keys[:where], keys[where + 1:]]) @ last * scale
    target = (others.max() / math.log(2) - below) * math.log(2) / scale
    k = (last * target / (last @ last)).to(dtype)
    assert torch.isfinite(k).all()
    cache.write(0, where, k.view(1, 1, D), cache.values[0][where:where + 1])
    desc = eg.make_attn_desc(1, 1, D, dtype)

    def run():
        out = torch.full_like(q, float("nan"))
        eg.engram_attn_paged(desc, q, cu_of([q_len]), cache.kv_len, cache.table, cache.k, cache.v, out, q_len)
        assert eg.engram_check_errors() == 0
        return f64(out)
    clean = run()
    page, slot = cache.place(0, where, 1)
    cache.v[page, slot, 0, 5] = float("inf")
    got = run()
    keep = np.arange(D) != 5
    np.testing.assert_allclose(got[-1, 0, keep], clean[-1, 0, keep], rtol=2.0 ** -7, atol=1e-6)
    x = got[-1, 0, 5]
    assert np.isposinf(x) if want == "inf" else np.isnan(x), x
    if where == N - 1:       # seen by the last row alone
        np.testing.assert_allclose(got[:-1], clean[:-1], rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_that_are_nowhere_finite(value, dtype):
    # every value of every tile, in prompts and chunks: the rare path for each of them, in time
    heads, kv_heads, d, lens = 8, 2, 128, [1000, 3, 260]
    total = sum(lens)
    q, k = randn((total, heads, d), 1, dtype), randn((total, kv_heads, d), 2, dtype)
    v = torch.full((total, kv_heads, d), value, dtype=dtype, device="cuda")
    desc = eg.make_attn_desc(heads, kv_heads, d, dtype)
    out = torch.zeros_like(q)
    eg.engram_attn_prompt(desc, q, k, v, cu_of(lens), out)
    assert eg.engram_check_errors() == 0
    o = f64(out)
    assert (np.isposinf(o) if value == float("inf") else np.isnan(o)).all()
    cache = Paged(lens, 16, kv_heads, d, dtype, 3)
    cache.v.fill_(value)
    for chunk in ([700, 3, 200], [1, 2, 4]):
        q, out = q[:sum(chunk)], torch.zeros_like(q[:sum(chunk)])
        eg.engram_attn_paged(desc, q, cu_of(chunk), cache.kv_len, cache.table, cache.k, cache.v, out, max(chunk))
        assert eg.engram_check_errors() == 0
        o = f64(out)
        assert (np.isposinf(o) if value == float("inf") else np.isnan(o)).all()
