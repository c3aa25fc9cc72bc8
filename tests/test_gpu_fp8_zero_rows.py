"""GPU: attention over an 8-bit cache in which some value rows are zeros. Such a row weighs in the softmax and adds
nothing, whatever its scale (the append gives it 1), so it takes nothing from the other rows' range: it counts as
one of scale 2^-92."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from oracle import kv_fp8
from oracle.attention import attend
from oracle.numerics import e4m3_to_f64
from tests.attn_helpers import STEP, UNIT, f64
from tests.fp8_helpers import PagedFp8, few_rows, run

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def put(cache, i, k, v, scale_of_zeros=None):
    """Sequence i's keys and values, quantised; `scale_of_zeros`: another byte for value rows of zeros."""
    (kc, ks), (vc, vs) = kv_fp8.quantise(k), kv_fp8.quantise(v)
    if scale_of_zeros is not None:
        vs = np.where((vc & 0x7F).any(-1), vs, scale_of_zeros).astype(np.uint8)
    cache.write(i, 0, kc, ks, vc, vs)
    cache.keys[i], cache.values[i] = kv_fp8.values(kc, ks), kv_fp8.values(vc, vs)
    cache.codes[i], cache.exponents[i] = e4m3_to_f64(vc), vs.astype(np.int64) - 127


def check(cache, i, q, out, lse, dtype, scale, rows):
    """The tolerance of the 8-bit tests (tests/fp8_helpers.py) but for what small contributions lose.

    Few rows: probabilities times their value's scale are rounded to f16 with the row's largest such product, in
    which rows of zeros count with 2^-92, at 2^11 or more, so that half of f16's smallest step, 2^-25, is at most 2^-36
    of it; times the key's codes, summed over the keys. More rows: in bf16 the largest probability is at 2^-24 or more,
    and it or its product with a value may be flushed below 2^-126, in f16 at 2^6 or more, and it loses half a step of
    2^-24.
    """
    k, v, codes, exponents = cache.keys[i], cache.values[i], cache.codes[i], cache.exponents[i]
    qq, D = f64(q), k.shape[2]
    n, H, _ = qq.shape
    m, Hk, _ = k.shape
    want, want_lse, mass, dot, vsum = attend(qq, k, v, scale)
    few, u = few_rows(rows, D), UNIT[dtype]
    lost, small = np.zeros((n, H, D)), np.zeros((n, H))
    for t in range(n):
        seen = m - n + t + 1
        if seen <= 0:
            continue
        for h in range(H):
            c = h // (H // Hk)
            if few:
                w = np.exp(scale * (k[:seen, c] @ qq[t, h]) - want_lse[t, h])
                real = codes[:seen, c].any(-1)
                most = np.ldexp(w, np.where(real, exponents[:seen, c], -92)).max()
                lost[t, h] = 2.0 ** -36 * most * np.abs(codes[:seen, c]).sum(0)
                small[t, h] = 2.0 ** -39 * np.abs(qq[t, h]).max() * scale * np.abs(k[:seen, c]).sum(1).max()
            else:
                lost[t, h] = 2.0 ** -102 * (vsum[t, h] + seen) if dtype == BF16 else 2.0 ** -31 * vsum[t, h]
    e = (D + 6) * 2.0 ** -24 * dot + small + 2.0 ** -21 * (1 + dot / 16)
    tol = ((2.0 ** -11 if few else u) + 2 * e + 2.0 ** -16)[..., None] * mass + lost
    tol += u * (np.abs(want) + tol) + STEP[dtype]
    off = np.abs(f64(out) - want)
    assert (off <= tol).all(), f"{(off > tol).sum()} of {off.size} outputs off, worst {np.max(off / tol):.3g} of the tolerance"
    got, empty = f64(lse), np.isneginf(want_lse)
    assert (np.isneginf(got) == empty).all(), "lse is -inf exactly where a row sees nothing"
    got, want_lse = np.where(empty, 0.0, got), np.where(empty, 0.0, want_lse)
    off = np.abs(got - want_lse)
    assert (off <= e + 2.0 ** -16 + 2.0 ** -22 * np.abs(want_lse)).all(), f"lse off by {off.max():.3g}"


#: tokens, query heads, key-value heads, head_dim, further columns of the page table (which decide whether two
#: key-value heads make an item): every form of either kernel.
FORMS = {
    "8 rows, 128": (1, 16, 2, 128, 2), "8 rows of two heads, 128": (1, 16, 2, 128, 2000),
    "16 rows, 128": (2, 16, 2, 128, 2), "16 rows of two heads, 128": (2, 16, 2, 128, 2000),
    "32 rows, 128": (4, 16, 2, 128, 2), "48 rows, 128": (6, 8, 1, 128, 2), "tiles, 128": (20, 8, 2, 128, 2),
    "8 rows, 64": (1, 16, 2, 64, 2), "8 rows of two heads, 64": (1, 16, 2, 64, 2000),
    "16 rows, 64": (2, 16, 2, 64, 2), "16 rows of two heads, 64": (2, 16, 2, 64, 2000),
    "32 rows, 64": (4, 16, 2, 64, 2), "48 rows, 64": (6, 8, 1, 64, 2), "64 rows, 64": (8, 8, 1, 64, 2),
    "tiles, 64": (30, 8, 2, 64, 2), "8 rows, 80": (1, 16, 2, 80, 2), "32 rows, 48": (4, 16, 2, 48, 2),
}

#: the values' sizes (an exponent), how far the zero rows' scores lie above the others' (log2), the scale byte of zeros
SIZES = {
    "small": (-36, 0.0, None), "smaller": (-60, 0.0, None), "sink": (-18, 18.4, None), "far sink": (-10, 60.0, None),
    "sink over ordinary values": (0, 40.0, None), "farthest sink": (-40, 90.0, None), "large": (30, 0.0, None),
    "larger": (90, -4.0, None), "another scale": (-30, 3.0, 200), "the smallest scale": (20, 1.0, 0),
}


def make(form, lens, exponent, above, byte, where, dtype, seed=3):
    tokens, heads, kv_heads, D, columns = form
    g = np.random.default_rng(seed)
    cache = PagedFp8(lens, 16, kv_heads, D, seed, columns=columns)
    q = g.standard_normal((tokens * len(lens), heads, D))
    q[..., 0] = 4.0
    q = torch.from_numpy(q).to(device="cuda", dtype=dtype)
    for i, n in enumerate(lens):
        k, v = g.standard_normal((2, n, kv_heads, D)) * 0.25
        k[..., 0] = 0.0
        v = np.ldexp(v, exponent)
        zeros = {"first": slice(0, 1), "middle": slice(n // 2, n // 2 + 2), "some": slice(1, n - 1, 7),
                 "last": slice(n - 1, n)}[where]
        v[zeros] = 0.0
        k[zeros, :, 0] = above * math.log(2.0) * D ** 0.5 / 4.0
        put(cache, i, k, v, byte)
    return cache, q


@pytest.mark.parametrize("where", ["first", "middle", "some", "last"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("form", ["8 rows, 128", "tiles, 128"])
def test_sizes_beside_zeros(form, size, where):
    run_case(FORMS[form], (700,), *SIZES[size], where, BF16)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("size", ["small", "sink"])
def test_every_form(form, size):
    run_case(FORMS[form], (40, 333), *SIZES[size], "some", BF16)


@pytest.mark.parametrize("form", ["16 rows, 128", "48 rows, 64", "tiles, 64"])
@pytest.mark.parametrize("exponent,above", [(-8, 0.0), (-4, 9.0)])
def test_f16(form, exponent, above):
    run_case(FORMS[form], (17, 260), exponent, above, None, "some", F16)


def run_case(form, lens, exponent, above, byte, where, dtype):
    tokens, heads, kv_heads, D, _ = form
    cache, q = make(form, lens, exponent, above, byte, where, dtype)
    _, out, lse = run(cache, [tokens] * len(lens), heads, D, dtype, q=q)
    assert eg.engram_check_errors() == 0
    for i in range(len(lens)):
        s = slice(i * tokens, (i + 1) * tokens)
        check(cache, i, q[s], out[s], lse[s], dtype, D ** -0.5, tokens * heads // kv_heads)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("exponent", [-20, -30])
def test_columns_of_small_values(form, exponent):
    """Rows that have ordinary values in the even columns alone, and as many with small values in the odd ones: what
    those columns hold is lost only below 2^-36 of the ordinary rows' products."""
    tokens, heads, kv_heads, D, _ = FORMS[form]
    cache, q = make(FORMS[form], (450,), 0, 0.0, None, "some", BF16)
    v = cache.values[0].copy()
    v[0::2, :, 1::2] = 0.0
    v[1::2, :, 0::2] = 0.0
    v[1::2] = np.ldexp(v[1::2], exponent)
    put(cache, 0, cache.keys[0], v)
    _, out, lse = run(cache, [tokens], heads, D, BF16, q=q)
    assert eg.engram_check_errors() == 0
    check(cache, 0, q, out, lse, BF16, D ** -0.5, tokens * heads // kv_heads)


@pytest.mark.parametrize("form", ["8 rows, 128", "16 rows of two heads, 64", "48 rows, 128", "tiles, 64"])
def test_nothing_but_zeros(form):
    """Outputs are zeros; the logarithm of the sum is as ever."""
    tokens, heads, kv_heads, D, _ = FORMS[form]
    cache, q = make(FORMS[form], (300,), 0, 0.0, None, "some", BF16)
    put(cache, 0, cache.keys[0], np.zeros_like(cache.values[0]))
    _, out, lse = run(cache, [tokens], heads, D, BF16, q=q)
    assert eg.engram_check_errors() == 0 and (out == 0).all()
    check(cache, 0, q, out, lse, BF16, D ** -0.5, tokens * heads // kv_heads)
