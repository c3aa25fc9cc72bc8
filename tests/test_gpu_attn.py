"""GPU: attention over packed prompts and over a paged cache, and the cache's append, against the
float64 oracle, within tolerances derived in attn_helpers.tolerance."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from deepseek_v4_engram_gb300 import _lib
from tests.attn_helpers import Paged, assert_attn_close, cu_of, f64, randn, reference

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def nan_like(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def run_prompt(lens, heads, kv_heads, head_dim, dtype, seed=1, q_scale=1.0, scale=None, fused=True,
               edit=None, stream=None):
    """Runs the operator; returns q, k, v, out and lse."""
    total = sum(lens)
    qkv = randn((total, heads + 2 * kv_heads, head_dim), seed, dtype)
    qkv[:, :heads] *= q_scale
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    if not fused:
        q = q.contiguous()
        k = k.transpose(0, 1).contiguous().transpose(0, 1)     # heads outermost
        v = v.contiguous()
    if edit is not None:
        edit(q, k, v)
    desc = eg.make_attn_desc(heads, kv_heads, head_dim, dtype, scale)
    out, lse = nan_like((total, heads, head_dim), dtype), torch.full((total, heads), 7.0, device="cuda")
    eg.engram_attn_prompt(desc, q, k, v, cu_of(lens), out, lse_out=lse, stream=stream)
    if stream is None:
        assert eg.engram_check_errors() == 0
    return q, k, v, out, lse


def check_prompt(lens, heads, kv_heads, head_dim, dtype, **kw):
    q, k, v, out, lse = run_prompt(lens, heads, kv_heads, head_dim, dtype, **kw)
    scale = kw.get("scale") or 1 / math.sqrt(head_dim)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        assert_attn_close(out[s], lse[s], reference(q[s], k[s], v[s], scale), dtype, head_dim, scale)
        at += n


@pytest.mark.parametrize("lens", [[1], [2], [17], [127], [128], [129], [255, 1, 256, 257],
                                  [0, 5, 0, 0, 40, 0], [300, 1, 64, 0, 127, 513], [1100]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_lengths(lens, dtype):
    check_prompt(lens, 8, 2, 128, dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (6, 2), (10, 2), (14, 2), (16, 1),
                                            (9, 1), (32, 8)])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_prompt_head_layouts(heads, kv_heads, head_dim):
    check_prompt([70, 1, 333], heads, kv_heads, head_dim, BF16, seed=3)


@pytest.mark.parametrize("head_dim", [8, 24, 56, 72, 80, 96, 120])
def test_prompt_odd_widths(head_dim):
    check_prompt([150, 29], 6, 2, head_dim, F16, seed=4)


@pytest.mark.parametrize("heads,kv_heads", [(17, 1), (64, 2), (100, 1), (128, 1)])
def test_many_heads_share_a_key(heads, kv_heads):
    check_prompt([70, 1, 5], heads, kv_heads, 64, BF16, seed=16)
    check_paged([1, 2, 9], [5, 300, 1031], 16, heads, kv_heads, 128, F16, seed=16)


def test_prompt_separate_buffers_and_orders():
    check_prompt([260, 31], 8, 4, 64, BF16, seed=5, fused=False)


@pytest.mark.parametrize("q_scale,scale", [(40.0, None), (1.0, 1e-3), (4.0, 1.0)])
def test_prompt_sharp_and_flat_softmax(q_scale, scale):
    check_prompt([400], 4, 1, 64, BF16, seed=6, q_scale=q_scale, scale=scale)


def test_prompt_scores_that_grow_along_the_keys():
    # every tile raises the maximum, by far more than rounding hides
    def edit(q, k, v):
        n = k.shape[0]
        q.fill_(0.25)
        k.copy_((torch.arange(n, device="cuda") * 0.05)[:, None, None].expand_as(k).to(k.dtype))
    check_prompt([900], 4, 2, 64, F16, seed=7, edit=edit)


@pytest.mark.parametrize("head_dim", [64, 128])
def test_prompt_values_nobody_may_see(head_dim):
    # infinities and NaN in keys and values reach the rows that see them and no others: neither the
    # rows before them nor the sequences beside them in the buffer
    lens, bad = [200, 77, 300], 200 + 40
    where = [(200 + 40, "k", float("nan")), (277 + 130, "v", float("inf")), (277 + 290, "v", float("nan"))]

    def edit(q, k, v):
        for t, which, x in where:
            (k if which == "k" else v)[t, 0, head_dim // 2] = x
    clean = run_prompt(lens, 8, 2, head_dim, BF16, seed=8)
    _, _, _, out, lse = run_prompt(lens, 8, 2, head_dim, BF16, seed=8, edit=edit)
    o, c = f64(out), f64(clean[3])
    # other key-value heads and sequence 0 are untouched
    np.testing.assert_array_equal(o[:, 4:], c[:, 4:])
    np.testing.assert_array_equal(o[:200], c[:200])
    # sequence 1: rows before the NaN key are as they were, the others are NaN
    np.testing.assert_array_equal(o[200:240, :4], c[200:240, :4])
    assert np.isnan(o[240:277, :4]).all() and np.isnan(f64(lse)[240:277, :4]).all()
    # sequence 2: column d is +inf from the infinity on and NaN from the NaN on, the rest finite
    d = head_dim // 2
    keep = np.arange(head_dim) != d
    np.testing.assert_allclose(o[277:, :4][:, :, keep], c[277:, :4][:, :, keep], rtol=2 ** -7, atol=1e-6)
    np.testing.assert_allclose(o[277:407, :4, d], c[277:407, :4, d], rtol=2 ** -7, atol=1e-6)
    assert np.isposinf(o[407:567, :4, d]).all() and np.isnan(o[567:, :4, d]).all()


def test_prompt_tokens_of_no_sequence_stay():
    desc = eg.make_attn_desc(2, 1, 64, BF16)
    q, k, v = (randn((50, h, 64), 9 + h, BF16) for h in (2, 1, 1))
    out = torch.full((50, 2, 64), 3.0, dtype=BF16, device="cuda")
    cu = torch.tensor([5, 25, 30], dtype=torch.int32, device="cuda")
    eg.engram_attn_prompt(desc, q, k, v, cu, out)
    o = f64(out)
    assert (o[:5] == 3).all() and (o[30:] == 3).all()
    for s in (slice(5, 25), slice(25, 30)):
        assert_attn_close(out[s], None, reference(q[s], k[s], v[s], 0.125), BF16, 64, 0.125)


def test_prompt_boundaries_beyond_the_tensor_are_cut():
    desc = eg.make_attn_desc(2, 1, 64, BF16)
    q, k, v = (randn((40, h, 64), 19 + h, BF16) for h in (2, 1, 1))
    out = nan_like((40, 2, 64), BF16)
    cu = torch.tensor([-9, 10, 7, 4000], dtype=torch.int32, device="cuda")   # [0,10) [10,10) [7,40)
    eg.engram_attn_prompt(desc, q, k, v, cu, out)
    torch.cuda.synchronize()
    assert_attn_close(out[10:], None, tuple(r[3:] for r in reference(q[7:], k[7:], v[7:], 0.125)),
                      BF16, 64, 0.125)


def run_paged(cache, q_lens, heads, head_dim, dtype, seed=2, max_q=None, stream=None, workspace=None):
    kv_heads = cache.k.shape[2]
    q = randn((sum(q_lens), heads, head_dim), seed, dtype)
    desc = eg.make_attn_desc(heads, kv_heads, head_dim, dtype)
    out = nan_like(q.shape, dtype)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    eg.engram_attn_paged(desc, q, cu_of(q_lens), cache.kv_len, cache.table, cache.k, cache.v, out,
                         max(q_lens) if max_q is None else max_q, workspace=workspace, lse_out=lse,
                         stream=stream)
    return q, out, lse


def check_paged(q_lens, kv_lens, page, heads, kv_heads, head_dim, dtype, seed=2, layout="nhd", **kw):
    cache = Paged(kv_lens, page, kv_heads, head_dim, dtype, seed, layout)
    q, out, lse = run_paged(cache, q_lens, heads, head_dim, dtype, seed, **kw)
    assert eg.engram_check_errors() == 0
    scale, at = 1 / math.sqrt(head_dim), 0
    for i, n in enumerate(q_lens):
        s = slice(at, at + n)
        assert_attn_close(out[s], lse[s], reference(q[s], cache.keys[i], cache.values[i], scale),
                          dtype, head_dim, scale)
        at += n


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 256])
@pytest.mark.parametrize("head_dim,dtype", [(128, BF16), (64, F16)])
def test_decode_pages(page, head_dim, dtype):
    check_paged([1] * 6, [1, 127, 128, 129, 700, 1999], page, 8, 2, head_dim, dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 7), (6, 2), (16, 1), (32, 8), (13, 1)])
def test_decode_head_layouts(heads, kv_heads):
    check_paged([1, 1, 1], [5, 300, 1031], 16, heads, kv_heads, 128, BF16, seed=3)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
@pytest.mark.parametrize("q_lens", [[1, 1], [4, 3], [200, 31]])
def test_cache_layouts(layout, q_lens):
    check_paged(q_lens, [517, 60], 16, 8, 4, 80, BF16, seed=4, layout=layout)


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([5, 5, 5], [5, 6, 900]),              # a whole prompt, one more, a draft over a long cache
    ([300, 1, 0, 64], [300, 2000, 50, 1064]),
    ([129, 257], [1000, 257]),
    ([3, 2, 7], [0, 1, 5]),                # caches shorter than the chunk: rows that see nothing
    ([300, 200], [10, 0]),
    ([1, 1], [0, 0]),
])
@pytest.mark.parametrize("heads,kv_heads,dtype", [(8, 2, BF16), (3, 1, F16)])
def test_chunks(q_lens, kv_lens, heads, kv_heads, dtype):
    check_paged(q_lens, kv_lens, 32, heads, kv_heads, 128, dtype, seed=5)


def test_long_cache_is_shared_between_sms():
    check_paged([1, 1], [40000, 3], 64, 4, 2, 64, BF16, seed=6)
    check_paged([6], [30001], 48, 8, 1, 128, F16, seed=6)
    check_paged([90], [9001], 16, 4, 1, 128, BF16, seed=6)


def test_max_q_only_picks_the_kernel():
    # a longer chunk than max_q says, and a shorter one
    check_paged([70, 2], [300, 9], 16, 8, 2, 64, BF16, seed=7, max_q=1)
    check_paged([1, 2], [300, 9], 16, 8, 2, 64, BF16, seed=7, max_q=500)


@pytest.mark.parametrize("q_len", [1, 4, 100])
def test_cache_values_that_only_later_rows_see(q_len):
    cache = Paged([400], 16, 1, 64, BF16, 8)
    clean = run_paged(cache, [q_len], 2, 64, BF16, 9)
    cache.v[cache.place(0, 399, 1) + (0, 5)] = float("inf")       # seen by the last row alone
    _, out, _ = run_paged(cache, [q_len], 2, 64, BF16, 9)
    o, c = f64(out), f64(clean[1])
    np.testing.assert_allclose(o[:-1], c[:-1], rtol=2 ** -7, atol=1e-4)
    assert np.isposinf(o[-1, :, 5]).all()
    keep = np.arange(64) != 5
    np.testing.assert_allclose(o[-1][:, keep], c[-1][:, keep], rtol=2 ** -7, atol=1e-6)


def test_offsets_past_32_bits():
    # 2^32 elements of keys: pages at both ends and in the middle of the cache
    pages, page, kv_heads, d = 65540, 64, 8, 128
    k = torch.empty((pages, page, kv_heads, d), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    ids = [65539, 0, 32768, 65538, 1]
    n = 5 * 64 - 3
    kk, vv = randn((320, kv_heads, d), 1, BF16), randn((320, kv_heads, d), 2, BF16)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    desc = eg.make_attn_desc(16, kv_heads, d, BF16)
    eg.engram_kv_append(desc, kk[:n], vv[:n], cu_of([n]), kv_len, table, k, v)
    for j, p in enumerate(ids):
        m = min(64, n - 64 * j)
        assert torch.equal(k[p, :m], kk[64 * j:64 * j + m]) and torch.equal(v[p, :m], vv[64 * j:64 * j + m])
    for q_len in (1, 40):
        q = randn((q_len, 16, d), 3, BF16)
        out = nan_like(q.shape, BF16)
        eg.engram_attn_paged(desc, q, cu_of([q_len]), kv_len, table, k, v, out, q_len)
        scale = 1 / math.sqrt(d)
        assert_attn_close(out, None, reference(q, kk[:n], vv[:n], scale), BF16, d, scale)
    assert eg.engram_check_errors() == 0


@pytest.mark.parametrize("page,layout,head_dim,dtype", [(16, "nhd", 128, BF16), (24, "hnd", 72, F16),
                                                        (8, "pair", 8, BF16)])
def test_append(page, layout, head_dim, dtype):
    q_lens, kv_lens, kv_heads = [3, 0, 1, 40, 70], [10, 9, 300, 40, 61], 3
    cache = Paged(kv_lens, page, kv_heads, head_dim, dtype, 11, layout)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    kv = randn((sum(q_lens), 2 * kv_heads, head_dim), 12, dtype)
    k, v = kv[:, :kv_heads], kv[:, kv_heads:]
    at = 0
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):
        skip = max(0, n - m)      # tokens before position 0 are not kept
        p = cache.place(i, m - n + skip, n - skip)
        want_k[p], want_v[p] = k[at + skip:at + n], v[at + skip:at + n]
        at += n
    desc = eg.make_attn_desc(kv_heads, kv_heads, head_dim, dtype)
    eg.engram_kv_append(desc, k, v, cu_of(q_lens), cache.kv_len, cache.table, cache.k, cache.v)
    assert eg.engram_check_errors() == 0
    bits = torch.int16      # slots that nobody owns hold NaN
    assert torch.equal(cache.k.contiguous().view(bits), want_k.contiguous().view(bits))
    assert torch.equal(cache.v.contiguous().view(bits), want_v.contiguous().view(bits))


def test_bad_pages_and_lengths_are_reported():
    cache = Paged([100, 40], 16, 2, 64, BF16, 13)
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    table = cache.table.clone()
    table[0, 1] = cache.k.shape[0]
    table[1, 0] = -1
    q, k = randn((2, 4, 64), 1, BF16), randn((2, 2, 64), 2, BF16)
    out = nan_like(q.shape, BF16)
    for max_q in (1, 64):
        eg.engram_attn_paged(desc, q, cu_of([1, 1]), cache.kv_len, table, cache.k, cache.v, out, max_q)
        assert eg.engram_check_errors() == _lib.DEVERR_PAGE_RANGE
        assert np.isfinite(f64(out)).all()
    before = cache.k.clone()
    bad = torch.full_like(table, 1 << 30)
    eg.engram_kv_append(desc, k, k, cu_of([1, 1]), cache.kv_len, bad, cache.k, cache.v)
    assert eg.engram_check_errors() == _lib.DEVERR_PAGE_RANGE
    long = torch.tensor([16 * table.shape[1] + 1, 40], dtype=torch.int32, device="cuda")
    eg.engram_kv_append(desc, k[:1], k[:1], cu_of([1, 0]), long, cache.table, cache.k, cache.v)
    assert eg.engram_check_errors() == _lib.DEVERR_CACHE_FULL
    assert torch.equal(before.view(torch.int16), cache.k.view(torch.int16))
    full = torch.zeros_like(table)          # pages for every position of the table
    clean = torch.zeros_like(cache.k)
    eg.engram_attn_paged(desc, q, cu_of([1, 1]), long, full, clean, clean, out, 1)
    assert eg.engram_check_errors() == _lib.DEVERR_CACHE_FULL


def test_empty_calls_write_nothing():
    desc = eg.make_attn_desc(2, 1, 64, BF16)
    e = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    kv = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    eg.engram_attn_prompt(desc, e, kv, kv, cu_of([0, 0]), e.clone())
    cache = Paged([10], 16, 1, 64, BF16, 1)
    eg.engram_attn_paged(desc, e, cu_of([0]), cache.kv_len, cache.table, cache.k, cache.v, e.clone(), 1)
    eg.engram_kv_append(desc, kv, kv, cu_of([0]), cache.kv_len, cache.table, cache.k, cache.v)
    assert eg.engram_check_errors() == 0


def test_other_streams_and_a_reused_workspace():
    # two streams with a workspace each, calls in a row that reuse it without waiting
    cache = Paged([9000, 700], 64, 2, 128, BF16, 14)
    desc = eg.make_attn_desc(8, 2, 128, BF16)
    want1 = run_paged(cache, [1, 1], 8, 128, BF16, 3)[1:]
    want2 = run_paged(cache, [40, 9], 8, 128, BF16, 4)[1:]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(eg.engram_attn_workspace_size(desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = []
    for rep in range(6):
        i = rep % 2
        with torch.cuda.stream(streams[i]):
            got.append(run_paged(cache, [1, 1], 8, 128, BF16, 3, workspace=ws[i])[1:] + want1)
            got.append(run_paged(cache, [40, 9], 8, 128, BF16, 4, workspace=ws[i], stream=streams[i])[1:] + want2)
    torch.cuda.synchronize()
    for out, lse, want_out, want_lse in got:
        assert torch.equal(out, want_out) and torch.equal(lse, want_lse)   # and the same bits each time


def test_a_default_workspace_on_another_stream():
    # The call waits behind work on its stream; what is allocated and written on the current one in the
    # meantime, of the workspace's very size, must not be its workspace.
    cache = Paged([9000, 700], 64, 2, 128, BF16, 14)
    desc = eg.make_attn_desc(8, 2, 128, BF16)
    want = run_paged(cache, [40, 9], 8, 128, BF16, 4)[1:]
    size, stream = eg.engram_attn_workspace_size(desc), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    q, cu, out = randn((49, 8, 128), 4, BF16), cu_of([40, 9]), nan_like((49, 8, 128), BF16)
    stream.wait_stream(torch.cuda.current_stream())
    eg.engram_attn_paged(desc, q, cu, cache.kv_len, cache.table, cache.k, cache.v, out, 40, stream=stream)
    for _ in range(3):
        torch.empty(size, dtype=torch.uint8, device="cuda").zero_()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])


def test_inside_a_cuda_graph():
    cache = Paged([300, 77], 16, 2, 64, BF16, 15)
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    q, kv = randn((2, 4, 64), 1, BF16), randn((2, 2, 64), 2, BF16)
    out, cu = nan_like(q.shape, BF16), cu_of([1, 1])
    ws = torch.empty(eg.engram_attn_workspace_size(desc), dtype=torch.uint8, device="cuda")

    def step():
        eg.engram_kv_append(desc, kv, kv, cu, cache.kv_len, cache.table, cache.k, cache.v)
        eg.engram_attn_paged(desc, q, cu, cache.kv_len, cache.table, cache.k, cache.v, out, 1, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6):       # new inputs and one position less each time
        q.copy_(randn(q.shape, seed, BF16))
        kv.copy_(randn(kv.shape, seed + 10, BF16))
        cache.kv_len -= 1
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            m = int(cache.kv_len[i])
            keys, values = cache.keys[i][:m].clone(), cache.values[i][:m].clone()
            keys[-1], values[-1] = kv[i], kv[i]
            assert_attn_close(out[i:i + 1], None, reference(q[i:i + 1], keys, values, 0.125), BF16, 64, 0.125)
    assert eg.engram_check_errors() == 0


def test_python_refusals():
    desc = eg.make_attn_desc(4, 2, 64, BF16)
    q, k = randn((5, 4, 64), 1, BF16), randn((5, 2, 64), 2, BF16)
    out, cu = torch.empty_like(q), cu_of([5])

    def prompt(**kw):
        a = dict(q=q, k=k, v=k, cu_seqlens=cu, out=out)
        a.update(kw)
        eg.engram_attn_prompt(desc, **a)
    for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(k=k[:4]), dict(k=k.float()), dict(v=q),
                dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu.cpu()), dict(q=q.cpu()), dict(out=out[:4]),
                dict(q=torch.empty((5, 64, 4), dtype=BF16, device="cuda").transpose(1, 2)),
                dict(lse_out=torch.empty((5, 3), device="cuda")), dict(cu_seqlens=cu[:0]),
                dict(workspace=torch.empty(10, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            prompt(**bad)
    with pytest.raises(eg.EngramError, match="workspace"):
        prompt(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(eg.EngramError, match="overlaps"):
        prompt(out=q)
    with pytest.raises(eg.EngramError, match="strides"):
        wide = torch.empty((5, 4, 68), dtype=BF16, device="cuda")
        prompt(q=wide[:, :, :64])
    with pytest.raises(eg.EngramError, match="strides"):
        prompt(k=k[:, :1].expand(-1, 2, -1))
    cache = Paged([10], 16, 2, 64, BF16, 1)
    for bad in (dict(kv_len=cache.kv_len.long()), dict(block_table=cache.table[:0]), dict(k_cache=cache.k[0]),
                dict(v_cache=cache.v[:, :8]), dict(kv_len=cu)):
        a = dict(kv_len=cache.kv_len, block_table=cache.table, k_cache=cache.k, v_cache=cache.v)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            eg.engram_attn_paged(desc, q, cu, out=out, max_q=5, **a)
        with pytest.raises((ValueError, TypeError)):
            eg.engram_kv_append(desc, k, k, cu, **a)
    with pytest.raises(TypeError):
        eg.make_attn_desc(4, 2, 64, torch.float32)
