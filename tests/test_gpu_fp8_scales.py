"""GPU: attention over an 8-bit cache whose values are near the ends of what its format and its type hold."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from oracle import kv_fp8
from oracle.numerics import e4m3_to_f64
from tests.fp8_helpers import PagedFp8, assert_close, reference, run

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def put_values(cache, codes, scales):
    """Sequence 0's values as bytes."""
    kc, ks = kv_fp8.quantise(cache.keys[0])
    cache.write(0, 0, kc, ks, codes, scales)
    cache.values[0] = kv_fp8.values(codes, scales)
    cache.codes[0], cache.exponents[0] = e4m3_to_f64(codes), scales.astype(np.int64) - 127


@pytest.mark.parametrize("low", [160, 243, 254])
@pytest.mark.parametrize("tokens,heads,head_dim,m", [
    (1, 8, 128, 700), (2, 8, 64, 700), (4, 8, 128, 300), (6, 8, 128, 300), (8, 8, 64, 500), (40, 8, 128, 128),
    (70, 2, 64, 100)])
def test_the_largest_scales(tokens, heads, head_dim, m, low):
    """Bytes up to 254, beside smaller ones and by themselves. (Over one key tile where rows are many.)"""
    g = np.random.default_rng(low)
    cache = PagedFp8([m], 16, 1, head_dim, 5)
    scales = g.integers(low, 255, (m, 1)).astype(np.uint8)
    codes = (g.integers(0x10, 0x30, (m, 1, head_dim)) | g.integers(0, 2, (m, 1, head_dim)) * 128).astype(np.uint8)   # < 0.5
    put_values(cache, codes, scales)
    q, out, lse = run(cache, [tokens], heads, head_dim, BF16)
    assert eg.engram_check_errors() == 0
    scale = head_dim ** -0.5
    assert_close(out, lse, *reference(cache, 0, q, scale), BF16, head_dim, scale, tokens * heads)


@pytest.mark.parametrize("tokens", [1, 5, 60])
@pytest.mark.parametrize("exponent", [98, -90])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_large_and_small_values_whose_scores_grow(tokens, exponent, head_dim):
    """Maxima that grow by 2^80 from the first key to the last, evenly, so that as much as there may be lies
    between a sum's base and its largest term."""
    m = 1500
    cache = PagedFp8([m], 16, 2, head_dim, 6)
    g = np.random.default_rng(7)
    k = np.zeros((m, 2, head_dim))
    k[..., 0] = (np.arange(m) * (80 * math.log(2) / m))[:, None] / 4
    kc, ks = kv_fp8.quantise(k)
    vc, vs = kv_fp8.quantise(np.ldexp(g.uniform(-1.9, 1.9, (m, 2, head_dim)), exponent))
    cache.write(0, 0, kc, ks, vc, vs)
    cache.keys[0], cache.values[0] = kv_fp8.values(kc, ks), kv_fp8.values(vc, vs)
    cache.codes[0], cache.exponents[0] = e4m3_to_f64(vc), vs.astype(np.int64) - 127
    q = torch.zeros((tokens, 4, head_dim), dtype=BF16, device="cuda")
    q[..., 0] = 4.0
    _, out, lse = run(cache, [tokens], 4, head_dim, BF16, q=q, scale=1.0)
    assert eg.engram_check_errors() == 0
    assert_close(out, lse, *reference(cache, 0, q, 1.0), BF16, head_dim, 1.0, tokens * 2)
