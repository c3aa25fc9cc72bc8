"""Host-side checks of the 8-bit cache's operators (no GPU): what the C ABI and the binding refuse."""
import ctypes
import types

import pytest
import torch

from deepseek_v4_engram_gb300 import _lib, attn, attn_fp8, build
from tests.test_attn_devices import On, on

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
    c = dict(k=0x1000000, v=0x2000000, k_scale=0x3000000, v_scale=0x4000000, k_page_stride=2048, k_slot_stride=128,
             k_head_stride=64, v_page_stride=2048, v_slot_stride=128, v_head_stride=64, k_scale_page_stride=32,
             k_scale_head_stride=16, v_scale_page_stride=32, v_scale_head_stride=16, n_pages=8, page_size=16,
             block_table=0x8000, table_width=4)
    c.update(kw)
    return ctypes.byref(_lib.EngramKvCacheFp8(**c))


KV = dict(k=view(0x40000, 128), v=view(0x50000, 128))


def append(lib, d=desc(), k=KV["k"], v=KV["v"], cu=0x8800, n=2, total=9, kv_len=0x9000, c=cache()):
    return lib.engram_kv_append_fp8(d, k, v, cu, n, total, kv_len, c, None)


def read(lib, d=desc(), k=KV["k"], v=KV["v"], cu=0x8800, n=2, total=9, kv_len=0x9000, c=cache()):
    return lib.engram_kv_read_fp8(d, cu, n, total, kv_len, c, k, v, None)


def attend(lib, d=desc(), q=view(), cu=0x8800, n=2, total=9, max_q=5, kv_len=0x9000, c=cache(), out=view(0x900000),
           lse=None, ws=0x100000, size=WS):
    return lib.engram_attn_paged_fp8(d, q, cu, n, total, max_q, kv_len, c, out, lse, ws, size, None)


@pytest.mark.parametrize("bad,code", [
    (dict(n_heads=0), EINVAL), (dict(n_kv_heads=3), EINVAL), (dict(head_dim=0), EINVAL), (dict(dtype=2), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(head_dim=136), EUNSUPPORTED), (dict(head_dim=72), EUNSUPPORTED),
    (dict(n_heads=258, n_kv_heads=2), EUNSUPPORTED)])
@pytest.mark.parametrize("call", [append, read, attend])
def test_descriptor(lib, call, bad, code):
    assert call(lib, desc(**bad), n=0) == code      # even where there would be nothing to do


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None), dict(v=0x2000008),
    dict(k_scale=0x3000004), dict(n_pages=0), dict(table_width=0), dict(page_size=0), dict(k_slot_stride=0),
    dict(v_head_stride=72), dict(k_page_stride=-16), dict(k_scale_page_stride=24), dict(v_scale_head_stride=8),
    dict(v_page_stride=1 << 39)])
@pytest.mark.parametrize("call", [append, read, attend])
def test_cache(lib, call, bad):
    assert call(lib, c=cache(**bad)) == EINVAL, bad
    assert lib.engram_last_error()


@pytest.mark.parametrize("call", [append, read, attend])
def test_sizes(lib, call):
    assert call(lib, c=None) == EINVAL
    assert call(lib, c=cache(page_size=24)) == EUNSUPPORTED
    assert call(lib, c=cache(page_size=1 << 20, table_width=1 << 11)) == EUNSUPPORTED
    assert call(lib, kv_len=None) == EINVAL and call(lib, kv_len=0x9001) == EINVAL
    assert call(lib, cu=None) == EINVAL and call(lib, cu=0x8102) == EINVAL
    assert call(lib, n=-1) == EINVAL and call(lib, total=-1) == EINVAL
    assert call(lib, total=1 << 24) == EUNSUPPORTED
    assert call(lib, n=0) == OK and call(lib, total=0) == OK       # nothing to do


@pytest.mark.parametrize("call", [append, read])
def test_rows(lib, call):
    for bad in (dict(k=None), dict(v=view(0x50004, 128)), dict(k=view(0x40000, 100)), dict(v=view(0x50000, 0))):
        assert call(lib, **bad) == EINVAL, bad


def test_attention_arguments(lib):
    def refused(word, **kw):
        assert attend(lib, **kw) == EINVAL
        assert word in lib.engram_last_error().decode()
    refused("q", q=None)
    refused("aligned", q=view(0x10008))
    refused("strides", out=view(0x900000, 260))
    refused("max_q", max_q=-1)
    refused("workspace", ws=None)
    refused("workspace", ws=0x100010)
    refused("workspace", size=64)
    refused("lse", lse=0x902)


@pytest.mark.parametrize("word,change", [
    ("out overlaps q", dict(out=view(0x10000 + 2 * 64))),
    ("out overlaps the cache", dict(out=view(0x1000000 + 2048 * 3))),
    ("out overlaps the cache", dict(out=view(0x2000000 + 64))),
    ("out overlaps the cache's scales", dict(out=view(0x3000000 + 240))),
    ("out overlaps kv_len", dict(out=view(0x9000 - 512))),
    ("lse overlaps the cache's scales", dict(lse=0x4000000 + 32)),
    ("lse overlaps block_table", dict(lse=0x8000 + 8)),
    ("workspace overlaps the cache", dict(ws=0x1000000 - 256)),
    ("rows overlap", dict(out=view(0x900000, 512, 8))),
])
def test_attention_overlap(lib, word, change):
    assert attend(lib, **change) == EINVAL
    assert word in lib.engram_last_error().decode()


@pytest.mark.parametrize("word,change", [
    ("the cache overlaps k", dict(k=view(0x1000000 + 64, 128))),
    ("scales overlaps v", dict(v=view(0x4000000 + 16, 128))),
    ("the cache overlaps the cache", dict(c=cache(v=0x1000000 + 128))),
    ("scales overlaps the cache", dict(c=cache(k_scale=0x1000000 + 256))),
    ("the cache overlaps cu_seqlens", dict(cu=0x1000000 + 2048)),
    ("scales overlaps kv_len", dict(kv_len=0x3000000)),
    ("rows overlap", dict(c=cache(k_slot_stride=64))),          # slots on top of each other's heads
    ("rows overlap", dict(c=cache(v_scale_page_stride=16))),
])
def test_append_overlap(lib, word, change):
    assert append(lib, **change) == EINVAL
    got = lib.engram_last_error().decode()
    assert word in got, got


@pytest.mark.parametrize("word,change", [
    ("k_out overlaps the cache", dict(k=view(0x1000000 + 64, 128))),
    ("v_out overlaps the cache's scales", dict(v=view(0x4000000 + 16, 128))),
    ("v_out overlaps k_out", dict(v=view(0x40000 + 64 * 2, 128))),
    ("k_out overlaps cu_seqlens", dict(k=view(0x8800, 128))),
    ("v_out overlaps kv_len", dict(v=view(0x9000, 128))),
    ("rows overlap", dict(k=view(0x40000, 64))),
])
def test_read_overlap(lib, word, change):
    assert read(lib, **change) == EINVAL
    got = lib.engram_last_error().decode()
    assert word in got, got


def test_packed_cache_is_laid_out_as_the_structure():
    values = [(i + 1) << 40 for i in range(4)] + list(range(1, 13)) + [9 << 40, 14]
    assert bytes(_lib.EngramKvCacheFp8(*values)) == _lib.PACK_CACHE_FP8.pack(*values)


# ---- the binding: tensors that only say where they are, and a library that counts calls

@pytest.fixture
def calls(monkeypatch):
    made = []

    def entry(name):
        return lambda *a: made.append((name, a[-1])) or 0
    names = ("engram_kv_append_fp8", "engram_kv_read_fp8", "engram_attn_paged_fp8")
    fake = types.SimpleNamespace(engram_attn_workspace_size=lambda d: 64, **{n: entry(n) for n in names})
    for module in (attn, attn_fp8):
        monkeypatch.setattr(module, "lib", lambda: fake)
    monkeypatch.setattr(attn, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(attn, "_raw_stream", lambda device: 1000 + device)
    return made


DESC = attn.make_attn_desc(4, 2, 64)
BF16 = torch.bfloat16
NAMES = {"engram_kv_append_fp8": "k v cu_seqlens kv_len block_table k_cache v_cache k_scale v_scale",
         "engram_kv_read_fp8": "cu_seqlens kv_len block_table k_cache v_cache k_scale v_scale k_out v_out",
         "engram_attn_paged_fp8": "q cu_seqlens kv_len block_table k_cache v_cache k_scale v_scale out workspace "
                                  "lse_out"}


def arguments(name):
    a = {n: on((5, h, 64), BF16) for n, h in {"q": 4, "out": 4, "k": 2, "v": 2, "k_out": 2, "v_out": 2}.items()}
    a["cu_seqlens"], a["kv_len"] = on(3, torch.int32), on(2, torch.int32)
    a["block_table"] = on((2, 4), torch.int32)
    a["k_cache"], a["v_cache"] = (on((8, 16, 2, 64), torch.uint8) for _ in range(2))
    a["k_scale"], a["v_scale"] = (on((8, 2, 16), torch.uint8) for _ in range(2))
    a["workspace"], a["lse_out"] = on(64, torch.uint8), on((5, 4), torch.float32)
    a = {n: a[n] for n in NAMES[name].split()}
    if name == "engram_attn_paged_fp8":
        a["max_q"] = 3
    return a


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_has_to_be_on_the_current_device(calls, name):
    call, a = getattr(attn_fp8, name), arguments(name)
    call(DESC, **a)
    call(DESC, stream=types.SimpleNamespace(cuda_stream=77, device_index=0), **a)
    assert calls == [(name, 1000), (name, 77)]
    for n, t in a.items():
        if not isinstance(t, On):
            continue
        with pytest.raises(ValueError, match="cuda:1"):
            call(DESC, **dict(a, **{n: on(t.shape, t.dtype, 1)}))
        with pytest.raises(ValueError):          # and a CPU tensor
            call(DESC, **dict(a, **{n: torch.zeros(t.shape, dtype=t.dtype)}))
    with pytest.raises(ValueError, match="current device"):
        call(DESC, **{n: on(t.shape, t.dtype, 1) if isinstance(t, On) else t for n, t in a.items()})
    with pytest.raises(ValueError, match="stream"):
        call(DESC, stream=types.SimpleNamespace(cuda_stream=77, device_index=1), **a)
    assert len(calls) == 2


@pytest.mark.parametrize("name", NAMES)
def test_shapes_and_types(calls, name):
    call, a = getattr(attn_fp8, name), arguments(name)
    wrong = {"k_cache": [on((8, 16, 2, 64), BF16), on((8, 16, 2, 32), torch.uint8), on((8, 2, 16, 64), torch.uint8),
                         on((8, 16, 2, 128), torch.uint8)[..., ::2], on((8, 16, 2, 64), torch.int8), None],
             "v_cache": [on((7, 16, 2, 64), torch.uint8)],
             "k_scale": [on((8, 16, 2), torch.uint8), on((8, 2, 16), torch.float32), on((8, 16, 2), torch.uint8).transpose(1, 2)],
             "v_scale": [on((8, 2, 15), torch.uint8)],
             "block_table": [on((3, 4), torch.int32), on((2, 4), torch.int64), on((2, 8), torch.int32)[:, ::2]],
             "kv_len": [on(3, torch.int32), on(2, torch.int64)],
             "cu_seqlens": [on(3, torch.int64), on(0, torch.int32)]}
    for n, tensors in wrong.items():
        for t in tensors:
            if isinstance(t, On):
                t.at = 0
            with pytest.raises((ValueError, TypeError)):
                call(DESC, **dict(a, **{n: t}))
    assert not calls
    call(DESC, **a)
    eight = dict(a)
    for n in ("k_cache", "v_cache"):
        eight[n] = on((8, 16, 2, 64), torch.float8_e4m3fn)
    for n in ("k_scale", "v_scale"):
        eight[n] = on((8, 2, 16), torch.float8_e8m0fnu)
    call(DESC, **eight)
    with pytest.raises(ValueError):
        call(DESC, **dict(eight, v_cache=a["v_cache"]))      # keys and values alike
    assert len(calls) == 2
