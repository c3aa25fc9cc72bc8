"""GPU: quantising a chunk's keys and values into an 8-bit cache, and reading positions back, bit for bit
against the float64 oracle."""
import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from deepseek_v4_engram_gb300 import _lib
from oracle import kv_fp8
from tests.attn_helpers import cu_of, f64
from tests.fp8_helpers import PagedFp8, assert_close, reference, rows

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def append(cache, k, v, q_lens, dtype, kv_len=None, table=None, **kw):
    desc = eg.make_attn_desc(k.shape[1], k.shape[1], k.shape[2], dtype)
    eg.engram_kv_append_fp8(desc, k, v, cu_of(q_lens), cache.kv_len if kv_len is None else kv_len,
                            cache.table if table is None else table, *cache.tensors, **kw)


def read(cache, q_lens, dtype, kv_len=None, table=None, fill=7.0, cu=None, **kw):
    kv_heads, d = cache.k.shape[2:]
    total = sum(q_lens)
    both = torch.full((total, 2 * kv_heads, d), fill, dtype=dtype, device="cuda")   # one buffer, beside each other
    k, v = both[:, :kv_heads], both[:, kv_heads:]
    desc = eg.make_attn_desc(kv_heads, kv_heads, d, dtype)
    eg.engram_kv_read_fp8(desc, cu_of(q_lens) if cu is None else cu, cache.kv_len if kv_len is None else kv_len,
                          cache.table if table is None else table, *cache.tensors, k, v, **kw)
    return k, v


def snapshot(cache):
    return [t.clone() for t in cache.tensors]


def expect(cache, want, i, start, k, v):
    """The rows k and v [n, heads, D] of sequence i from position start on, in the arrays `want`."""
    page, slot = cache.place(i, start, k.shape[0])
    for at, x in ((0, k), (1, v)):
        codes, scales = kv_fp8.quantise(f64(x))
        want[at][page, slot] = torch.from_numpy(codes).cuda()
        want[at + 2][page, :, slot] = torch.from_numpy(scales).cuda()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("head_dim", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page,layout,kv_heads", [(16, "nhd", 3), (48, "hnd", 1), (64, "pool", 8)])
def test_append(dtype, head_dim, page, layout, kv_heads):
    q_lens, kv_lens = [3, 0, 1, 40, 70], [10, 9, 300, 40, 61]
    cache = PagedFp8(kv_lens, page, kv_heads, head_dim, 11, layout)
    want = snapshot(cache)
    kv = rows((sum(q_lens), 2 * kv_heads, head_dim), 12, dtype, 3.0).cuda()
    k, v = kv[:, :kv_heads], kv[:, kv_heads:]
    at = 0
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):
        skip = max(0, n - m)      # tokens before position 0 are not kept
        expect(cache, want, i, m - n + skip, k[at + skip:at + n], v[at + skip:at + n])
        at += n
    append(cache, k, v, q_lens, dtype)
    assert eg.engram_check_errors() == 0
    for got, w in zip(cache.tensors, want):
        assert torch.equal(got, w)


def test_rows_of_every_kind():
    """Zeros, signed zeros, the largest values, values around a scale's border, subnormals, infinities and NaN."""
    d = 64
    for dtype in (BF16, F16):
        big = torch.finfo(dtype).max
        tiny = torch.finfo(dtype).tiny
        x = torch.zeros((16, 1, d), dtype=torch.float64)
        x[1, 0, ::2] = -0.0
        x[2, 0, 0], x[2, 0, 1] = big, -1.0
        x[3] = big
        x[4, 0, 3] = 448.0
        x[5, 0, 3] = 450.0
        x[6] = torch.linspace(-448, 448, d, dtype=torch.float64)
        x[7] = torch.linspace(0, 2.0 ** -6, d, dtype=torch.float64) * 448     # codes below the normal ones
        x[7, 0, 0] = 448.0
        x[8] = tiny / 4
        x[9] = torch.linspace(-1, 1, d, dtype=torch.float64) * tiny
        x[10, 0, 5] = float("inf")
        x[11, 0, 6] = -float("inf")
        x[12, 0, 7] = float("nan")
        x[13] = torch.tensor([17.0, 18, 19, 21, 23, 25, 27, 29] * (d // 8), dtype=torch.float64)   # ties to even
        x[14] = float("nan")
        x[15, 0, 63] = -(2.0 ** -14)
        x = x.to(dtype).cuda()
        cache = PagedFp8([16], 16, 1, d, 5)
        want = snapshot(cache)
        expect(cache, want, 0, 0, x, x.flip(0))
        append(cache, x, x.flip(0), [16], dtype)
        for got, w in zip(cache.tensors, want):
            assert torch.equal(got, w)
        k, v = read(cache, [16], dtype)
        bad = torch.tensor([i in (10, 11, 12, 14) for i in range(16)], device="cuda")
        assert torch.isnan(k[bad]).all() and torch.isfinite(k[~bad]).all()
        assert torch.isnan(v.flip(0)[bad]).all() and torch.isfinite(v.flip(0)[~bad]).all()
        assert torch.equal(k[0], x[0]) and torch.equal(k[1].view(torch.int16), x[1].view(torch.int16))
        assert eg.engram_check_errors() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("head_dim,page,layout", [(16, 16, "pool"), (64, 48, "nhd"), (80, 32, "hnd"), (128, 128, "nhd")])
def test_read(dtype, head_dim, page, layout):
    q_lens, kv_lens = [10, 0, 1, 299, 70, 5], [10, 9, 300, 300, 61, 0]
    cache = PagedFp8(kv_lens, page, 2, head_dim, 21, layout, dtype=dtype)
    k, v = read(cache, q_lens, dtype)
    assert eg.engram_check_errors() == 0
    at = 0
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):
        for got, rows_ in ((k, cache.keys[i]), (v, cache.values[i])):
            want = np.zeros((n, 2, head_dim))
            have = min(n, m)
            if have:
                want[n - have:] = rows_[m - have:]
            np.testing.assert_array_equal(f64(got[at:at + n]), f64(torch.from_numpy(want).to(dtype)))
        at += n


def test_read_rounds_once_and_stays_finite():
    # values that the type does not reach (scales of a bf16 append, for f16) are rounded, and cut at its largest
    cache = PagedFp8([64], 64, 1, 32, 3)
    g = np.random.default_rng(0)
    codes = g.integers(0, 127, (64, 1, 32)).astype(np.uint8) | (g.integers(0, 2, (64, 1, 32)).astype(np.uint8) << 7)
    scales = np.linspace(0, 254, 64).astype(np.uint8)[:, None]
    cache.write(0, 0, codes, scales, codes, scales)
    want = kv_fp8.values(codes, scales)
    for dtype in (F16, BF16):
        k, v = read(cache, [64], dtype)
        top = torch.finfo(dtype).max
        # 64 -> 32 -> 16 bits are one rounding: codes times a power of two, from 2^-100 on, are exact in f32
        expect_ = torch.from_numpy(np.clip(want, -top, top)).to(torch.float32).to(dtype)
        assert torch.equal(k.cpu(), expect_) and torch.equal(v.cpu(), expect_)


def test_read_back_what_was_appended():
    q_lens, kv_lens = [5, 17, 1], [5, 100, 33]
    cache = PagedFp8(kv_lens, 16, 2, 128, 7)
    k, v = (rows((23, 2, 128), s, BF16, 2.0).cuda() for s in (1, 2))
    append(cache, k, v, q_lens, BF16)
    for got, x in zip(read(cache, q_lens, BF16), (k, v)):
        top = f64(x.abs().amax(-1))[..., None]
        # half a step of a code: 2^-4 of a value, or of the smallest codes' step where it is far below the row's largest
        assert (np.abs(f64(got) - f64(x)) <= np.maximum(2.0 ** -4 * np.abs(f64(x)), 2.0 ** -17 * top)).all()
    assert eg.engram_check_errors() == 0


def test_errors_and_rows_of_no_sequence():
    cache = PagedFp8([100, 40], 16, 2, 64, 13)
    k = rows((2, 2, 64), 2, BF16).cuda()
    before = snapshot(cache)
    for bad_page in (cache.k.shape[0], -1, 1 << 30):
        bad = torch.full_like(cache.table, bad_page)
        append(cache, k, k, [1, 1], BF16, table=bad)
        assert eg.engram_check_errors() == _lib.DEVERR_PAGE_RANGE
        got = read(cache, [1, 1], BF16, table=bad)
        assert eg.engram_check_errors() == _lib.DEVERR_PAGE_RANGE
        assert not any(x.any() for x in got)
    long = torch.tensor([16 * cache.table.shape[1] + 1, 40], dtype=torch.int32, device="cuda")
    append(cache, k[:1], k[:1], [1, 0], BF16, kv_len=long)
    assert eg.engram_check_errors() == _lib.DEVERR_CACHE_FULL
    assert not any(x.any() for x in read(cache, [1, 0], BF16, kv_len=long))
    assert eg.engram_check_errors() == _lib.DEVERR_CACHE_FULL
    short = torch.tensor([-5, 0], dtype=torch.int32, device="cuda")      # empty caches: nothing is kept
    append(cache, k, k, [1, 1], BF16, kv_len=short)
    assert not any(x.any() for x in read(cache, [1, 1], BF16, kv_len=short))
    assert eg.engram_check_errors() == 0
    for got, w in zip(cache.tensors, before):
        assert torch.equal(got, w)
    # tokens of no sequence are neither written to the cache nor to the output; boundaries are cut
    cu = torch.tensor([2, 4, 100], dtype=torch.int32, device="cuda")
    k, v = read(cache, [5, 4], BF16, cu=cu)
    assert (k[:2] == 7).all() and (v[:2] == 7).all()
    np.testing.assert_array_equal(f64(k[2:4]), cache.keys[0][98:])
    np.testing.assert_array_equal(f64(v[4:]), cache.values[1][35:])
    assert eg.engram_check_errors() == 0


def test_empty_calls_write_nothing():
    cache = PagedFp8([10], 16, 1, 64, 1)
    e = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    append(cache, e, e, [0], BF16)
    read(cache, [0], BF16)
    assert eg.engram_check_errors() == 0


def test_offsets_past_32_bits():
    # 2^32 bytes of codes: pages at both ends and in the middle of the cache
    pages, page, kv_heads, d = 65540, 64, 8, 128
    k = torch.empty((pages, page, kv_heads, d), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.empty((pages, kv_heads, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    ids, n = [65539, 0, 32768, 65538, 1], 5 * 64 - 3
    kk, vv = rows((n, kv_heads, d), 1, BF16).cuda(), rows((n, kv_heads, d), 2, BF16).cuda()
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    desc = eg.make_attn_desc(16, kv_heads, d, BF16)
    eg.engram_kv_append_fp8(desc, kk, vv, cu_of([n]), kv_len, table, k, v, ks, vs)
    ko, vo = torch.empty_like(kk), torch.empty_like(vv)
    eg.engram_kv_read_fp8(desc, cu_of([n]), kv_len, table, k, v, ks, vs, ko, vo)
    for codes, scales, got, x in ((k, ks, ko, kk), (v, vs, vo, vv)):
        c, s = kv_fp8.quantise(f64(x))
        for j, p in enumerate(ids):
            m = min(64, n - 64 * j)
            assert torch.equal(codes[p, :m].cpu(), torch.from_numpy(c[64 * j:64 * j + m]))
            assert torch.equal(scales[p, :, :m].cpu(), torch.from_numpy(s[64 * j:64 * j + m].T.copy()))
        np.testing.assert_array_equal(f64(got), kv_fp8.values(c, s))
    scale = d ** -0.5
    for q_len in (1, 40):       # the few-row kernel and the tiled one
        q = torch.randn((q_len, 16, d), device="cuda").to(BF16)
        out = torch.empty_like(q)
        eg.engram_attn_paged_fp8(desc, q, cu_of([q_len]), kv_len, table, k, v, ks, vs, out, q_len)
        vc, ve = kv_fp8.quantise(f64(vv))
        held = PagedFp8.__new__(PagedFp8)
        held.keys, held.values = [kv_fp8.values(*kv_fp8.quantise(f64(kk)))], [kv_fp8.values(vc, ve)]
        held.codes, held.exponents = [kv_fp8.e4m3_to_f64(vc)], [ve.astype(np.int64) - 127]
        assert_close(out, None, *reference(held, 0, q, scale), BF16, d, scale, q_len * 2)
    assert eg.engram_check_errors() == 0
