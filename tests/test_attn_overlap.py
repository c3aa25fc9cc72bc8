"""Host checks that the attention operators refuse what they write over what they read (no GPU): parts
of one buffer that interleave are told apart from parts that share bytes."""
import ctypes

import pytest

from deepseek_v4_engram_gb300 import _lib, build

EINVAL = _lib.ENGRAM_EINVAL
H, HK, D, T = 8, 2, 64, 9
ROW = (2 * H + 2 * HK) * D          # a buffer of q, k, v and out beside each other, per token
Q = 0x100000
K, V, OUT = Q + 2 * H * D, Q + 2 * (H + HK) * D, Q + 2 * (H + 2 * HK) * D
WS, LSE = 0x4000000, 0x200000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def view(ptr, token=ROW, head=D):
    return ctypes.byref(_lib.EngramAttnView(ptr, token, head))


def desc():
    return ctypes.byref(_lib.EngramAttnDesc(H, HK, D, 0, 0.125))


@pytest.mark.parametrize("word,change", [
    ("out overlaps q", dict(out=view(Q + 2 * D))),                       # by a head, inside the buffer
    ("out overlaps q", dict(out=view(Q + 2 * 7 * D))),                   # its last head
    ("out overlaps v", dict(out=view(OUT - 2 * 8))),                     # by eight columns
    ("out overlaps k", dict(out=view(K + 2 * D))),
    ("out overlaps q", dict(out=view(OUT + 2 * 8 * D))),                 # into the next token's row
    ("out overlaps q", dict(out=view(Q, ROW * T // 3, D))),
    ("rows overlap", dict(out=view(0x900000, ROW, 8))),                  # heads on top of each other
    ("rows overlap", dict(out=view(0x900000, 4 * D))),                   # tokens on top of each other
    ("lse overlaps q", dict(lse=Q + 64)),
    ("lse overlaps out", dict(lse=OUT + 64)),
    ("lse overlaps cu_seqlens", dict(lse=0x8008)),
    ("lse overlaps workspace", dict(lse=WS + 1024)),
    ("workspace overlaps q", dict(ws=Q)),
    ("workspace overlaps out", dict(out=view(WS + 256 * 3, H * D))),
    ("workspace overlaps cu_seqlens", dict(cu=WS + 8)),
])
def test_prompt(lib, word, change):
    a = dict(q=view(Q), k=view(K), v=view(V), cu=0x8000, out=view(OUT), lse=LSE, ws=WS)
    a.update(change)
    assert lib.engram_attn_prompt(desc(), a["q"], a["k"], a["v"], a["cu"], 2, T, a["out"], a["lse"], a["ws"], 1 << 30,
                                  None) == EINVAL
    got = lib.engram_last_error().decode()
    assert word in got, got


CACHE = 0x1000000


@pytest.mark.parametrize("word,change", [
    ("out overlaps q", dict(out=view(Q + 2 * D))),
    ("out overlaps the cache", dict(out=view(CACHE + 2 * 2048 * 3, H * D))),
    ("out overlaps the cache", dict(out=view(CACHE + 2 * 1024, 4096))),       # the values' part of the pages
    ("out overlaps kv_len", dict(kv_len=OUT + 4)),
    ("out overlaps block_table", dict(table=OUT + 2 * ROW + 4)),
    ("lse overlaps kv_len", dict(lse=0x9004)),
    ("lse overlaps block_table", dict(lse=0xA000)),
    ("lse overlaps the cache", dict(lse=CACHE + 4)),
    ("workspace overlaps the cache", dict(ws=CACHE)),
    ("rows overlap", dict(out=view(0x900000, 8))),
])
def test_paged(lib, word, change):
    # keys and values in turn in one array of pages [8, 2, 16, HK, D]
    a = dict(q=view(Q), cu=0x8000, kv_len=0x9000, table=0xA000, out=view(OUT), lse=LSE, ws=WS)
    a.update(change)
    page = 16 * HK * D
    c = _lib.EngramKvCache(CACHE, CACHE + 2 * page, 2 * page, HK * D, D, 2 * page, HK * D, D, 8, 16, a["table"], 4)
    for max_q in (1, 9):
        assert lib.engram_attn_paged(desc(), a["q"], a["cu"], 2, T, max_q, a["kv_len"], ctypes.byref(c), a["out"],
                                     a["lse"], a["ws"], 1 << 30, None) == EINVAL
        assert word in lib.engram_last_error().decode()


def test_strides_beyond_any_address(lib):
    big = view(Q, (1 << 38) - 8)
    for a in (dict(q=big), dict(out=big)):
        v = dict(q=view(Q), out=view(OUT))
        v.update(a)
        assert lib.engram_attn_prompt(desc(), v["q"], view(K), view(V), 0x8000, 2, (1 << 24) - 1, v["out"], None, WS,
                                      1 << 30, None) == EINVAL
        assert "strides" in lib.engram_last_error().decode()
