"""GPU: cache lengths that no cache has, by the append as by the attention."""
import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from tests.attn_helpers import Paged, cu_of, f64, randn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H, HK, D = 4, 2, 64


@pytest.mark.parametrize("length", [-1, -(2 ** 31), -(2 ** 31) + 1])
def test_a_negative_length_is_an_empty_cache(length):
    # nothing kept, nothing seen, nothing reported
    cache = Paged([20, 9], 8, HK, D, BF16, 7)
    kv_len = torch.tensor([length, 9], dtype=torch.int32, device="cuda")
    desc, cu = eg.make_attn_desc(H, HK, D), cu_of([3, 1])
    k, q = randn((4, HK, D), 5, BF16), randn((4, H, D), 6, BF16)
    want = cache.k.clone()
    want[cache.place(1, 8, 1)] = k[3:]
    eg.engram_kv_append(desc, k, k, cu, kv_len, cache.table, cache.k, cache.v)
    assert eg.engram_check_errors() == 0
    assert torch.equal(cache.k.view(torch.int16), want.view(torch.int16))
    for max_q in (1, 64):
        out = torch.full_like(q, float("nan"))
        eg.engram_attn_paged(desc, q, cu, kv_len, cache.table, cache.k, cache.v, out, max_q)
        assert eg.engram_check_errors() == 0
        assert (f64(out[:3]) == 0).all() and np.isfinite(f64(out[3:])).all()
