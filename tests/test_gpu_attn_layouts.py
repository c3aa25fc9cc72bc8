"""GPU: outputs that lie between the queries, keys and values of one buffer, without sharing a byte with
them, against the float64 oracle; nothing else in the buffer changes."""
import math

import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from tests.attn_helpers import Paged, assert_attn_close, cu_of, randn, reference

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H, D, T = 4, 64, 150
SCALE = 1 / math.sqrt(D)

#: shape of the buffer, and its parts q, k, v and out as [T, H, D]
LAYOUTS = {
    "beside each other": ((T, 4 * H, D), lambda b: [b[:, i * H:(i + 1) * H] for i in range(4)]),
    "head by head": ((T, H, 4, D), lambda b: [b[:, :, i] for i in range(4)]),
    "heads outermost": ((H, T, 4, D), lambda b: [b[:, :, i].transpose(0, 1) for i in range(4)]),
    "parts between heads": ((H, 4, T, D), lambda b: [b[:, i].transpose(0, 1) for i in range(4)]),
    "columns of a wide head": ((T, H, 4 * D), lambda b: [b[..., i * D:(i + 1) * D] for i in range(4)]),
    "every other token": ((2 * T, 2 * H, D), lambda b: [b[::2, :H], b[::2, H:], b[1::2, :H], b[1::2, H:]]),
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_prompt(layout):
    shape, parts = LAYOUTS[layout]
    buffer = randn(shape, 3, BF16)
    q, k, v, out = parts(buffer)
    before, want = buffer.clone(), reference(q, k, v, SCALE)
    lse = torch.empty((T, H), device="cuda")
    eg.engram_attn_prompt(eg.make_attn_desc(H, H, D), q, k, v, cu_of([T]), out, lse_out=lse)
    assert eg.engram_check_errors() == 0
    assert_attn_close(out, lse, want, BF16, D, SCALE)
    for now, then in list(zip(parts(buffer), parts(before)))[:3]:
        assert torch.equal(now, then)
    # one head further it would be written over a part
    with pytest.raises(eg.EngramError, match="overlaps|rows"):
        eg.engram_attn_prompt(eg.make_attn_desc(H, H, D), q, k, v, cu_of([T]), k, lse_out=lse)


@pytest.mark.parametrize("n,max_q", [(1, 1), (7, 7), (7, 64)])
def test_output_beside_the_pages(n, max_q):
    # pages of keys, values and room for an output row between them
    cache = Paged([90], 16, H, D, BF16, 5)
    pool = torch.zeros((cache.k.shape[0], 3, 16, H, D), dtype=BF16, device="cuda")
    pool[:, 0], pool[:, 1] = cache.k, cache.v
    out = pool[:n, 2, 5]
    q = randn((n, H, D), 6, BF16)
    eg.engram_attn_paged(eg.make_attn_desc(H, H, D), q, cu_of([n]), cache.kv_len, cache.table, pool[:, 0], pool[:, 1],
                         out, max_q)
    assert eg.engram_check_errors() == 0
    assert_attn_close(out, None, reference(q, cache.keys[0], cache.values[0], SCALE), BF16, D, SCALE)
    with pytest.raises(eg.EngramError, match="overlaps the cache"):
        eg.engram_attn_paged(eg.make_attn_desc(H, H, D), q, cu_of([n]), cache.kv_len, cache.table, pool[:, 0],
                             pool[:, 1], pool[:n, 1, 5], max_q)
