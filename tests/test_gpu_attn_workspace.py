"""GPU: whose memory a call's default workspace is. It has to come from the pool of the call's stream:
the allocator hands memory on in the order of the stream that it was allocated on."""
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from deepseek_v4_engram_gb300 import attn
from tests.attn_helpers import Paged, cu_of, randn

pytestmark = pytest.mark.gpu


def test_default_workspace_belongs_to_the_calls_stream(monkeypatch):
    desc = eg.make_attn_desc(4, 2, 64)
    cache = Paged([300], 16, 2, 64, torch.bfloat16, 1)
    q, cu = randn((2, 4, 64), 2, torch.bfloat16), cu_of([2])
    out, size = torch.empty_like(q), eg.engram_attn_workspace_size(desc)
    side, taken, real = torch.cuda.Stream(), [], attn._scratch

    def spy(*a, **kw):
        ws = real(*a, **kw)
        taken.append(ws.data_ptr())
        return ws
    monkeypatch.setattr(attn, "_scratch", spy)

    def call(stream):
        del taken[:]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()       # so that no other free block has the workspace's size
        eg.engram_attn_paged(desc, q, cu, cache.kv_len, cache.table, cache.k, cache.v, out, 2, stream=stream)
        return taken[-1]               # the outermost call's

    def block():
        return torch.empty(size, dtype=torch.uint8, device="cuda")
    # what a call on the current stream gave back is what the next request there gets
    first = call(None)
    assert block().data_ptr() == first
    # a call on another stream: its memory goes to the next request on that stream, not to one here
    second = call(side)
    here = block()
    assert here.data_ptr() != second
    with torch.cuda.stream(side):
        assert block().data_ptr() == second
    torch.cuda.synchronize()
