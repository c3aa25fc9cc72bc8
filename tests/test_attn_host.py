"""Host-side checks of the attention operators' C ABI (no GPU), and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from deepseek_v4_engram_gb300 import _lib, build
from oracle.attention import attend

OK, EINVAL, EUNSUPPORTED = _lib.ENGRAM_OK, _lib.ENGRAM_EINVAL, _lib.ENGRAM_EUNSUPPORTED
WS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def desc(**kw):
    d = dict(n_heads=8, n_kv_heads=2, head_dim=64, dtype=0, scale=0.125)
    d.update(kw)
    return ctypes.byref(_lib.EngramAttnDesc(**d))


def view(ptr=0x10000, token=512, head=64):
    return ctypes.byref(_lib.EngramAttnView(ptr, token, head))


def cache(**kw):
    c = dict(k=0x1000000, v=0x2000000, k_page_stride=2048, k_slot_stride=128, k_head_stride=64,
             v_page_stride=2048, v_slot_stride=128, v_head_stride=64, n_pages=8, page_size=16,
             block_table=0x8000, table_width=4)
    c.update(kw)
    return ctypes.byref(_lib.EngramKvCache(**c))


@pytest.mark.parametrize("bad,code", [
    (dict(n_heads=0), EINVAL), (dict(n_kv_heads=3), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(head_dim=0), EINVAL), (dict(dtype=2), EINVAL), (dict(scale=0.0), EINVAL),
    (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(head_dim=136), EUNSUPPORTED), (dict(head_dim=68), EUNSUPPORTED),
    (dict(n_heads=258, n_kv_heads=2), EUNSUPPORTED)])
def test_descriptor(lib, bad, code):
    d = desc(**bad)
    assert lib.engram_attn_workspace_size(d) == 0
    # refused even where there would be nothing to do
    assert lib.engram_attn_prompt(d, view(), view(), view(), 16, 0, 0, view(), None, 256, WS, None) == code
    assert lib.engram_attn_paged(d, view(), 16, 0, 0, 1, 16, cache(), view(), None, 256, WS, None) == code
    assert lib.engram_kv_append(d, view(), view(), 16, 0, 0, 16, cache(), None) == code


def test_prompt_arguments(lib):
    def call(q=view(), k=view(0x40000, 128), v=view(0x50000, 128), cu=0x8000, n=2, total=9,
             out=view(0x900000), lse=None, ws=0x100000, size=WS, d=desc()):
        return lib.engram_attn_prompt(d, q, k, v, cu, n, total, out, lse, ws, size, None)

    def refused(word, **kw):
        assert call(**kw) == EINVAL
        assert word in lib.engram_last_error().decode()
    refused("q", q=None)
    refused("k", k=view(None))
    refused("aligned", q=view(0x10008))
    refused("strides", q=view(token=260))
    refused("strides", v=view(0x50000, 0))
    refused("strides", k=view(0x40000, 128, -64))
    refused("cu_seqlens", cu=None)
    refused("cu_seqlens", cu=0x8002)
    refused(">= 0", n=-1)
    refused(">= 0", total=-1)
    refused("overlaps q", out=view())
    refused("overlaps k", out=view(0x40000 - 512))
    refused("workspace", ws=None)
    refused("workspace", ws=0x100010)
    refused("workspace", size=64)
    refused("lse", lse=0x902)
    refused("desc", d=None)
    assert call(total=1 << 24) == EUNSUPPORTED
    assert call(q=None, total=0) == OK and call(q=None, n=0) == OK      # nothing to do
    # parts of one buffer interleave without overlapping
    assert call(q=view(0x10000, 1024), out=view(0x10000, 1024)) == EINVAL


def test_paged_arguments(lib):
    def call(q=view(), cu=0x8000, n=2, total=9, max_q=5, kv_len=0x9000, c=cache(), out=view(0x900000),
             ws=0x100000, size=WS):
        return lib.engram_attn_paged(desc(), q, cu, n, total, max_q, kv_len, c, out, None, ws, size, None)

    for bad in (dict(kv_len=None), dict(c=None), dict(c=cache(k=None)), dict(c=cache(v=0x2000008)),
                dict(c=cache(block_table=None)), dict(c=cache(n_pages=0)), dict(c=cache(table_width=0)),
                dict(c=cache(page_size=0)), dict(c=cache(k_slot_stride=0)), dict(c=cache(v_head_stride=60)),
                dict(c=cache(k_page_stride=-8)), dict(max_q=-1), dict(out=view(0x1000000)),
                dict(out=view(0x2000000 + 2048 * 2 * 7)), dict(size=0), dict(kv_len=0x9001)):
        assert call(**bad) == EINVAL, bad
        assert lib.engram_last_error()
    assert call(c=cache(page_size=12)) == EUNSUPPORTED
    assert call(c=cache(page_size=1 << 20, table_width=1 << 11)) == EUNSUPPORTED
    assert call(n=0) == OK and call(total=0) == OK


def test_append_arguments(lib):
    def call(k=view(0x40000, 128), v=view(0x50000, 128), c=cache(), kv_len=0x9000, total=9):
        return lib.engram_kv_append(desc(), k, v, 0x8000, 2, total, kv_len, c, None)
    for bad in (dict(k=None), dict(v=view(0x50004, 128)), dict(c=None), dict(kv_len=None),
                dict(k=view(0x40000, 100)), dict(c=cache(v_slot_stride=4))):
        assert call(**bad) == EINVAL, bad
    assert call(total=0) == OK


def test_workspace_grows_with_the_width(lib):
    n64 = lib.engram_attn_workspace_size(desc())
    n128 = lib.engram_attn_workspace_size(desc(head_dim=72))
    assert 0 < n64 < n128 == lib.engram_attn_workspace_size(desc(head_dim=128))


def test_oracle_against_softmax():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    out, lse, mass, dot, vsum = attend(q, k, v, 0.3)
    for t in range(5):
        for h in range(4):
            seen = 9 - 5 + t + 1
            s = 0.3 * torch.from_numpy(k[:seen, h // 2]) @ torch.from_numpy(q[t, h])
            w = torch.softmax(s, 0)
            np.testing.assert_allclose(out[t, h], (w @ torch.from_numpy(v[:seen, h // 2])).numpy(), rtol=1e-12)
            np.testing.assert_allclose(lse[t, h], torch.logsumexp(s, 0).item(), rtol=1e-12)
            assert (mass[t, h] >= np.abs(out[t, h]) - 1e-12).all()
    # rows that see nothing, and no keys at all
    out, lse, *_ = attend(q, k[:3], v[:3], 0.3)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    out, lse, *_ = attend(q, k[:0], v[:0], 0.3)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_packed_arguments_are_laid_out_as_the_structures():
    view = _lib.EngramAttnView(1 << 40, 2, 3)
    assert bytes(view) == _lib.PACK_VIEW.pack(1 << 40, 2, 3)
    values = [1 << 40, 2 << 40, 3, 4, 5, 6, 7, 8, 9, 10, 3 << 40, 11]
    assert bytes(_lib.EngramKvCache(*values)) == _lib.PACK_CACHE.pack(*values)
