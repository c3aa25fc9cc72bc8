"""GPU: attention over a paged cache in eight bits against the float64 oracle over the values that the
cache holds, within tolerances derived in fp8_helpers.tolerance."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from deepseek_v4_engram_gb300 import _lib
from oracle import kv_fp8
from tests.attn_helpers import cu_of, f64, randn
from tests.fp8_helpers import PagedFp8, assert_close, check, reference, rows, run

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("head_dim,dtype", [(128, BF16), (64, F16)])
def test_decode_pages(page, head_dim, dtype):
    check([1] * 6, [1, 127, 128, 129, 700, 1999], page, 8, 2, head_dim, dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 7), (6, 2), (16, 1), (32, 8), (13, 1), (9, 1), (17, 1), (33, 1),
                                            (64, 2), (100, 1), (128, 1)])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_decode_head_layouts(heads, kv_heads, head_dim):
    check([1, 1, 1], [5, 300, 1031], 16, heads, kv_heads, head_dim, BF16, seed=3)


@pytest.mark.parametrize("head_dim", [16, 32, 48, 80, 96, 112])
@pytest.mark.parametrize("q_lens", [[1, 1], [3, 2], [70, 5]])
def test_widths(head_dim, q_lens):
    check(q_lens, [517, 60], 16, 8, 4, head_dim, F16, seed=4)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "pool"])
@pytest.mark.parametrize("q_lens", [[1, 1], [4, 3], [200, 31]])
def test_cache_layouts(layout, q_lens):
    check(q_lens, [517, 60], 16, 8, 4, 80, BF16, seed=4, layout=layout)


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([5, 5, 5], [5, 6, 900]),              # a whole prompt, one more, a draft over a long cache
    ([300, 1, 0, 64], [300, 2000, 50, 1064]),
    ([129, 257], [1000, 257]),
    ([3, 2, 7], [0, 1, 5]),                # caches shorter than the chunk: rows that see nothing
    ([300, 200], [10, 0]),
    ([1, 1], [0, 0]),
    ([2, 1, 4], [-3, 1, 4]),               # a negative length is an empty cache
])
@pytest.mark.parametrize("heads,kv_heads,dtype", [(8, 2, BF16), (3, 1, F16)])
def test_chunks(q_lens, kv_lens, heads, kv_heads, dtype):
    check(q_lens, kv_lens, 32, heads, kv_heads, 128, dtype, seed=5)


@pytest.mark.parametrize("head_dim,dtype", [(64, BF16), (128, BF16), (128, F16), (64, F16)])
@pytest.mark.parametrize("q_lens,heads,kv_heads", [
    ([1, 1, 1], 4, 4), ([1, 1, 1], 20, 4), ([1, 1, 1], 2, 2), ([4, 1, 2], 8, 4), ([3, 0, 5], 6, 2), ([2, 2, 2], 32, 2),
    ([8, 3, 1], 8, 2), ([1, 1, 1], 64, 2)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_items_of_one_and_of_two_heads(q_lens, heads, kv_heads, head_dim, dtype, page):
    # an even number of heads that lie beside each other, few and many positions that the table could hold
    for columns in (2, 4000):
        check(q_lens, [517, 3, 1030], page, heads, kv_heads, head_dim, dtype, seed=6, columns=columns)
    # a cache that many items share, and one that ends in the middle of every part of a tile
    check(q_lens[:1], [9000 + 17 * kv_heads], page, heads, kv_heads, head_dim, dtype, seed=7, columns=4000)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows", [17, 31, 32, 33, 40, 47, 48, 49, 56, 63, 64, 65])
@pytest.mark.parametrize("head_dim", [48, 64, 128])
def test_rows_about_the_limits_of_the_kernels(rows, head_dim, dtype):
    # the rows of a key-value head as tokens, and as heads
    check([rows, 1, rows // 2], [rows + 500, 3, rows - 9], 48, 2, 2, head_dim, dtype, seed=11)
    check([1, 1, 1], [20001, 1, 130], 64, rows, 1, head_dim, dtype, seed=12)


@pytest.mark.parametrize("q_len", [3, 4, 6, 7, 9])
@pytest.mark.parametrize("group", [5, 7, 11])
@pytest.mark.parametrize("head_dim", [64, 112])
def test_tokens_whose_heads_two_warps_share(group, q_len, head_dim):
    check([q_len, 1, q_len - 1, 0, 2], [q_len, 1, 2000, 5, 129], 16, 2 * group, 2, head_dim, BF16, seed=13)


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("m", [1, 15, 16, 17, 31, 33, 63, 64, 65, 95, 97, 111, 127, 128, 129, 161, 191, 193, 255, 257])
def test_ends_inside_a_tile(m, head_dim):
    for q_len in (1, 3):
        check([q_len, 1], [m, 2], 16, 4, 2, head_dim, BF16, seed=9, columns=4000)
        check([q_len, 1], [m, 2], 16, 3, 1, head_dim, BF16, seed=9)


def test_long_cache_is_shared_between_sms():
    check([1, 1], [40000, 3], 64, 4, 2, 64, BF16, seed=6)
    check([6], [30001], 48, 8, 1, 128, F16, seed=6)
    check([30], [9001], 16, 4, 1, 128, BF16, seed=6)


def test_max_q_only_picks_the_kernel():
    # a longer chunk than max_q says, and a shorter one
    check([70, 2], [300, 9], 16, 8, 2, 64, BF16, seed=7, max_q=1)
    check([70, 2], [300, 9], 16, 8, 2, 64, BF16, seed=7, max_q=0)
    check([1, 2], [300, 9], 16, 8, 2, 64, BF16, seed=7, max_q=500)


@pytest.mark.parametrize("q_lens", [[1, 1], [40, 9], [3, 2]])
@pytest.mark.parametrize("spread", [8.0, 20.0])
def test_rows_of_very_different_sizes(q_lens, spread):
    # values whose scales differ by far more than their codes do; with small queries, so that scores stay apart
    check(q_lens, [400, 150], 16, 4, 2, 64, BF16, seed=8, spread=spread, q_scale=2.0 ** -spread)


@pytest.mark.parametrize("q_scale,scale", [(40.0, None), (1.0, 1e-3), (4.0, 1.0), (1e-30, None), (1e30, 1e-30)])
@pytest.mark.parametrize("q_lens", [[1, 3], [60, 50]])
def test_sharp_and_flat_softmax_and_sizes_of_queries(q_lens, q_scale, scale):
    check(q_lens, [400, 77], 16, 4, 1, 64, BF16, seed=6, q_scale=q_scale, scale=scale)


@pytest.mark.parametrize("q_len", [1, 5, 60])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scores_that_grow_along_the_keys(q_len, dtype):
    # every tile raises the maximum, by far more than rounding hides
    n, d = 900, 64
    cache = PagedFp8([n], 16, 2, d, 9)
    k = (torch.arange(n) * 0.05)[:, None, None].expand(n, 2, d)
    kc, ks = kv_fp8.quantise(f64(k))
    vc, vs = kv_fp8.quantise(cache.values[0])
    cache.write(0, 0, kc, ks, vc, vs)
    cache.keys[0] = kv_fp8.values(kc, ks)
    q = torch.full((q_len, 4, d), 0.25, dtype=dtype, device="cuda")
    _, out, lse = run(cache, [q_len], 4, d, dtype, q=q)
    assert_close(out, lse, *reference(cache, 0, q, 1 / math.sqrt(d)), dtype, d, 1 / math.sqrt(d), q_len * 2)
    assert eg.engram_check_errors() == 0


@pytest.mark.parametrize("q_len", [1, 4, 100])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_much_weight_in_small_probabilities(q_len, dtype):
    # one sharp key and a tail of keys 2^-16 of its weight that sums up to a visible share
    n, d = 20000, 64
    cache = PagedFp8([n], 64, 1, d, 10)
    q = torch.zeros((q_len, 1, d), dtype=dtype, device="cuda")
    q[:, :, 0] = 8.0
    k = np.zeros((n, 1, d))
    k[100, 0, 0] = 16 * math.log(2)      # scores: 8 * that / 8
    v = np.full((n, 1, d), 1.0)
    v[100] = -1.0
    parts = kv_fp8.quantise(k) + kv_fp8.quantise(v)
    cache.write(0, 0, *parts)
    cache.keys[0], cache.values[0] = kv_fp8.values(*parts[:2]), v
    cache.codes[0], cache.exponents[0] = v * 256, np.full((n, 1), -8)
    _, out, lse = run(cache, [q_len], 1, d, dtype, q=q)
    assert_close(out, lse, *reference(cache, 0, q, 1 / math.sqrt(d)), dtype, d, 1 / math.sqrt(d), q_len)


@pytest.mark.parametrize("where", ["scale", "code"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_len,at", [(1, 399), (4, 399), (4, 397), (10, 399), (10, 391), (20, 385), (28, 399), (28, 377),
                                      (100, 399), (100, 340), (100, 5)])
@pytest.mark.parametrize("columns", [2, 4000])
def test_nan_reaches_only_the_rows_that_see_it(q_len, at, which, where, columns):
    cache = PagedFp8([400], 16, 2, 64, 8, columns=columns)
    clean = run(cache, [q_len], 4, 64, BF16, 9)
    page, slot = cache.place(0, at, 1)
    if where == "scale":
        (cache.k_scale if which == "k" else cache.v_scale)[page, 0, slot] = 255
    else:
        (cache.k if which == "k" else cache.v)[page, slot, 0, 5] = 0xFF
    _, out, lse = run(cache, [q_len], 4, 64, BF16, 9)
    assert eg.engram_check_errors() == 0
    o, c = f64(out), f64(clean[1])
    first = max(0, at - (400 - q_len))     # the first row that sees it
    np.testing.assert_array_equal(o[:, 2:], c[:, 2:])     # the other key-value head's rows
    # another maximum or another way round may be taken for the rows before it
    np.testing.assert_allclose(o[:first], c[:first], rtol=2 ** -7, atol=1e-4)
    seen = o[first:, :2]
    if which == "k":
        assert np.isnan(seen).all() and np.isnan(f64(lse)[first:, :2]).all()
    elif where == "scale":
        assert np.isnan(seen).all() and np.isfinite(f64(lse)).all()
    else:
        assert np.isnan(seen[..., 5]).all()
        keep = np.arange(64) != 5
        np.testing.assert_allclose(seen[..., keep], c[first:, :2][..., keep], rtol=2 ** -7, atol=1e-4)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q_len", [1, 4, 10, 20, 28, 100])
@pytest.mark.parametrize("head_dim,dtype", [(64, BF16), (128, BF16), (128, F16)])
def test_not_finite_queries_stay_with_their_rows(q_len, bad, head_dim, dtype):
    cache = PagedFp8([400, 150], 16, 2, head_dim, 8)
    q, clean, lse = run(cache, [q_len, 3], 4, head_dim, dtype, 9)
    q[q_len // 2, 1, 5] = bad
    _, out, got = run(cache, [q_len, 3], 4, head_dim, dtype, q=q)
    assert eg.engram_check_errors() == 0
    o, c, row = f64(out), f64(clean), (q_len // 2, 1)
    assert np.isnan(o[row]).all() and np.isnan(f64(got)[row])
    o[row] = c[row]
    # another maximum may be taken for the rows beside it
    np.testing.assert_allclose(o, c, rtol=2 ** -7, atol=1e-4)
    others = np.ones(lse.shape, bool)
    others[row] = False
    np.testing.assert_allclose(f64(got)[others], f64(lse)[others], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("max_q", [1, 3, 64])
def test_tokens_of_no_sequence_stay(max_q):
    cache = PagedFp8([100, 40], 16, 1, 64, 3)
    q = randn((50, 2, 64), 9, BF16)
    out, lse = torch.full_like(q, 3.0), torch.full((50, 2), 3.0, device="cuda")
    cu = torch.tensor([5, 25, 30], dtype=torch.int32, device="cuda")
    desc = eg.make_attn_desc(2, 1, 64, BF16)
    eg.engram_attn_paged_fp8(desc, q, cu, cache.kv_len, cache.table, *cache.tensors, out, max_q, lse_out=lse)
    assert eg.engram_check_errors() == 0
    o = f64(out)
    assert (o[:5] == 3).all() and (o[30:] == 3).all() and (lse[:5] == 3).all() and (lse[30:] == 3).all()
    for i, s in enumerate((slice(5, 25), slice(25, 30))):
        assert_close(out[s], lse[s], *reference(cache, i, q[s], 0.125), BF16, 64, 0.125, max_q * 2)


@pytest.mark.parametrize("max_q", [1, 3, 64])
def test_bad_pages_and_lengths_are_reported(max_q):
    cache = PagedFp8([100, 40], 16, 2, 64, 13)
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    q = randn((2, 4, 64), 1, BF16)
    out, lse = torch.full_like(q, float("nan")), torch.empty((2, 4), device="cuda")
    cu = cu_of([1, 1])
    table = cache.table.clone()
    table[0, 1] = cache.k.shape[0]
    table[1, :3] = -1
    eg.engram_attn_paged_fp8(desc, q, cu, cache.kv_len, table, *cache.tensors, out, max_q, lse_out=lse)
    assert eg.engram_check_errors() == _lib.DEVERR_PAGE_RANGE
    # such positions read as zeros: keys of score 0 and values of 0
    cache.keys[0][16:32] = cache.values[0][16:32] = cache.codes[0][16:32] = 0
    assert_close(out[:1], lse[:1], *reference(cache, 0, q[:1], 0.125), BF16, 64, 0.125, max_q * 2)
    assert not out[1].any()
    np.testing.assert_allclose(f64(lse[1]), math.log(40), rtol=1e-5)
    full = torch.zeros_like(table)          # pages for every position of the table
    zero = [torch.zeros_like(t) for t in cache.tensors]
    long = torch.tensor([16 * table.shape[1] + 1, 40], dtype=torch.int32, device="cuda")
    eg.engram_attn_paged_fp8(desc, q, cu, long, full, *zero, out, max_q)
    assert eg.engram_check_errors() == _lib.DEVERR_CACHE_FULL
    assert not out.any()


def test_empty_calls_write_nothing():
    cache = PagedFp8([10], 16, 1, 64, 1)
    e = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    eg.engram_attn_paged_fp8(eg.make_attn_desc(2, 1, 64, BF16), e, cu_of([0]), cache.kv_len, cache.table,
                             *cache.tensors, e.clone(), 1)
    assert eg.engram_check_errors() == 0


def test_outputs_and_queries_with_strides():
    # queries inside a projection's output, outputs with heads outermost
    cache = PagedFp8([333, 20], 32, 2, 128, 5)
    for q_lens in ([1, 1], [40, 7]):
        n = sum(q_lens)
        wide = randn((n, 12, 128), 3, BF16)
        q = wide[:, 2:10]
        out = torch.full((8, n, 128), float("nan"), dtype=BF16, device="cuda").transpose(0, 1)
        desc = eg.make_attn_desc(8, 2, 128, BF16)
        eg.engram_attn_paged_fp8(desc, q, cu_of(q_lens), cache.kv_len, cache.table, *cache.tensors, out, max(q_lens))
        at = 0
        for i, m in enumerate(q_lens):
            s = slice(at, at + m)
            assert_close(out[s], None, *reference(cache, i, q[s], 128 ** -0.5), BF16, 128, 128 ** -0.5,
                         max(q_lens) * 4)
            at += m


def test_other_streams_and_a_reused_workspace():
    # two streams with a workspace each, calls in a row that reuse it without waiting
    cache = PagedFp8([9000, 700], 64, 2, 128, 14)
    desc = eg.make_attn_desc(8, 2, 128, BF16)
    want1 = run(cache, [1, 1], 8, 128, BF16, 3)[1:]
    want2 = run(cache, [40, 9], 8, 128, BF16, 4)[1:]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(eg.engram_attn_workspace_size(desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = []
    for rep in range(6):
        i = rep % 2
        with torch.cuda.stream(streams[i]):
            got.append(run(cache, [1, 1], 8, 128, BF16, 3, workspace=ws[i])[1:] + want1)
            got.append(run(cache, [40, 9], 8, 128, BF16, 4, workspace=ws[i], stream=streams[i])[1:] + want2)
    torch.cuda.synchronize()
    for out, lse, want_out, want_lse in got:
        assert torch.equal(out, want_out) and torch.equal(lse, want_lse)   # and the same bits each time


def test_appended_attended_and_read_back_inside_a_cuda_graph():
    """The three operators as a decoding step uses them, captured once and replayed on new tokens."""
    cache = PagedFp8([300, 77], 16, 2, 64, 15)
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    q = randn((2, 4, 64), 1, BF16)
    k, v = (rows((2, 2, 64), s, BF16).cuda() for s in (2, 3))
    out, cu = torch.full_like(q, float("nan")), cu_of([1, 1])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(eg.engram_attn_workspace_size(desc), dtype=torch.uint8, device="cuda")

    def step():
        paged = (cu, cache.kv_len, cache.table, *cache.tensors)
        eg.engram_kv_append_fp8(desc, k, v, *paged)
        eg.engram_attn_paged_fp8(desc, q, *paged, out, 1, workspace=ws)
        eg.engram_kv_read_fp8(desc, *paged, ko, vo)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6):       # new inputs and one position less each time
        q.copy_(randn(q.shape, seed, BF16))
        k.copy_(rows(k.shape, seed + 10, BF16))
        v.copy_(rows(v.shape, seed + 20, BF16))
        cache.kv_len -= 1
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            m = int(cache.kv_len[i])
            kc, ks = kv_fp8.quantise(f64(k[i:i + 1]))
            vc, vs = kv_fp8.quantise(f64(v[i:i + 1]))
            np.testing.assert_array_equal(f64(ko[i:i + 1]), kv_fp8.values(kc, ks))
            np.testing.assert_array_equal(f64(vo[i:i + 1]), kv_fp8.values(vc, vs))
            now = PagedFp8.__new__(PagedFp8)
            now.keys = [np.concatenate([cache.keys[i][:m - 1], kv_fp8.values(kc, ks)])]
            now.values = [np.concatenate([cache.values[i][:m - 1], kv_fp8.values(vc, vs)])]
            now.codes = [np.concatenate([cache.codes[i][:m - 1], kv_fp8.e4m3_to_f64(vc)])]
            now.exponents = [np.concatenate([cache.exponents[i][:m - 1], vs.astype(np.int64) - 127])]
            assert_close(out[i:i + 1], None, *reference(now, 0, q[i:i + 1], 0.125), BF16, 64, 0.125, 2)
    assert eg.engram_check_errors() == 0


def test_eight_bit_types_are_the_same_bytes():
    cache = PagedFp8([200], 16, 2, 64, 16)
    want = run(cache, [3], 4, 64, BF16, 3)[1]
    cache.k, cache.v = cache.k.view(torch.float8_e4m3fn), cache.v.view(torch.float8_e4m3fn)
    cache.k_scale, cache.v_scale = cache.k_scale.view(torch.float8_e8m0fnu), cache.v_scale.view(torch.float8_e8m0fnu)
    assert torch.equal(run(cache, [3], 4, 64, BF16, 3)[1], want)


def test_refusals():
    cache = PagedFp8([10], 16, 2, 64, 1)
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    q, cu = randn((5, 4, 64), 1, BF16), cu_of([5])
    args = (cu, cache.kv_len, cache.table, *cache.tensors)
    with pytest.raises(eg.EngramError, match="workspace"):
        eg.engram_attn_paged_fp8(desc, q, *args, torch.empty_like(q), 5,
                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(eg.EngramError, match="overlaps"):
        eg.engram_attn_paged_fp8(desc, q, *args, q, 5)
    with pytest.raises(eg.EngramError, match="multiple of 16"):
        odd = eg.make_attn_desc(4, 2, 72, BF16)
        wide = torch.empty((5, 4, 72), dtype=BF16, device="cuda")
        codes = torch.zeros((3, 16, 2, 72), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((3, 2, 16), dtype=torch.uint8, device="cuda")
        eg.engram_attn_paged_fp8(odd, wide, cu, cache.kv_len, cache.table, codes, codes, scales, scales,
                                 torch.empty_like(wide), 5)
    with pytest.raises(ValueError):
        eg.engram_attn_paged_fp8(desc, q.half(), *args, torch.empty_like(q), 5)
