"""GPU: attention over an 8-bit cache with scores so large that they differ by whole steps of f32: the key that is
ahead decides."""
import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from oracle import kv_fp8
from tests.attn_helpers import f64, randn
from tests.fp8_helpers import PagedFp8, run

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("tokens", [1, 3, 7, 40, 150])
@pytest.mark.parametrize("at", [0, 5, 100, 500, 640])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_far_key_decides(tokens, at, sign, dtype):
    """Scores of 2^26 and more, and one that is a quarter larger (or nearer to 0) than all others: its value is the
    result, exactly, since every other probability is 0 and that of the key 1."""
    m, d = 800, 64
    cache = PagedFp8([m], 16, 2, d, 4, dtype=dtype)
    k = np.zeros((m, 2, d))
    k[..., 0] = sign * 2.0 ** 14 * (1 if sign > 0 else 1.25)
    k[at, :, 0] = sign * 2.0 ** 14 * (1.25 if sign > 0 else 1)
    kc, ks = kv_fp8.quantise(k)
    np.testing.assert_array_equal(kv_fp8.values(kc, ks), k)
    vc, vs = kv_fp8.quantise(cache.values[0])
    cache.write(0, 0, kc, ks, vc, vs)
    q = torch.zeros((tokens, 4, d), dtype=dtype, device="cuda")
    q[..., 0] = 2.0 ** 12
    _, out, lse = run(cache, [tokens], 4, d, dtype, q=q, scale=1.0)
    assert eg.engram_check_errors() == 0
    want = torch.from_numpy(np.repeat(cache.values[0][at], 2, 0)).to(dtype)    # all rows see the key
    assert torch.equal(out.cpu(), want.expand_as(out.cpu()))
    score = sign * 2.0 ** 26 * (1.25 if sign > 0 else 1)
    np.testing.assert_allclose(f64(lse), score, rtol=2.0 ** -21)    # eight roundings to f32


@pytest.mark.parametrize("tokens", [1, 4, 60])
def test_far_keys_of_equal_scores_share(tokens):
    """Two keys of the same score, 2^25 and more, and of the same scale: the mean of their values, but for the
    roundings of a probability (2^-11 or, in tiles, none: it is a power of two) and of the result."""
    m, d = 400, 128
    cache = PagedFp8([m], 16, 1, d, 4)
    k = np.zeros((m, 1, d))
    k[..., 0] = 2.0 ** 15
    k[[3, 290], :, 0] = 1.5 * 2.0 ** 15
    v = f64(randn((m, 1, d), 8, BF16))
    v = np.where(np.abs(v).max(-1, keepdims=True) > 0, v / np.abs(v).max(-1, keepdims=True), v)
    (kc, ks), (vc, vs) = kv_fp8.quantise(k), kv_fp8.quantise(v)
    assert (vs == vs[0]).all()
    cache.write(0, 0, kc, ks, vc, vs)
    q = torch.zeros((tokens, 2, d), dtype=BF16, device="cuda")
    q[..., 0] = 2.0 ** 10
    _, out, lse = run(cache, [tokens], 2, d, BF16, q=q, scale=1.0)
    assert eg.engram_check_errors() == 0
    a, b = (kv_fp8.values(vc, vs)[i] for i in (3, 290))
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * (np.abs(a) + np.abs(b)) / 2
    assert (np.abs(f64(out) - (a + b) / 2) <= tol).all()
