"""GPU: what very small probabilities carry. Probabilities are rounded to the type of the values for
their product with them, while their sum keeps all bits: what the rounding loses is lost from the
result."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_engram_gb300 as eg
from tests.attn_helpers import STEP, UNIT, Paged, cu_of, f64, randn, reference, tolerance

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

#: Probabilities in f16 are kept in units of 2^-6 of the largest one at least (the tiled kernel; the
#: few-row kernel 2^-15): half the type's smallest step is then this much of it.
TAIL_STEP = {F16: STEP[F16] * 2.0 ** -6, BF16: STEP[BF16]}


def tail_tolerance(ref, dtype, head_dim, scale):
    """attn_helpers.tolerance with the smallest step that probabilities have in fact: there
    STEP * vsum stands for a probability's rounding near the type's smallest value, here
    TAIL_STEP * vsum. The rest of it, and the result's own rounding, are the same."""
    out, lse, mass, dot, vsum = ref
    full = tolerance(ref, dtype, head_dim, scale)[0]
    return full - (1 + UNIT[dtype]) * (STEP[dtype] - TAIL_STEP[dtype]) * vsum


def assert_tail_close(got, ref, dtype, head_dim, scale):
    t = tail_tolerance(ref, dtype, head_dim, scale)
    err = np.abs(f64(got) - ref[0])
    assert (err <= t).all(), f"worst {np.max(err / t):.3g} of the tolerance"


@pytest.mark.parametrize("max_q", [1, 64], ids=["few rows", "tiles"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_long_tail_behind_one_sharp_key(max_q, dtype):
    # One key far above 8191 others of 2^-25.6 of its weight each, which f16 cannot hold beside 1. Its
    # value is zero, so the tail is the whole result. 160 sequences: a CTA walks whole caches.
    n, seqs, d = 8192, 160, 64
    cache = Paged([n] * seqs, 64, 1, d, dtype, 31)
    scale = 1 / math.sqrt(d)
    sharp = 25.6 * math.log(2) / scale / d      # against queries of ones
    cache.k.zero_()
    for i in range(seqs):
        v = torch.rand((n, 1, d), device="cuda") * 64 + 32
        v[0] = 0
        v = v.to(dtype)
        k = torch.zeros((n, 1, d), dtype=dtype, device="cuda")
        k[0] = sharp
        cache.write(i, 0, k, v)
        cache.keys[i], cache.values[i] = k, v
    q = torch.ones((seqs, 1, d), dtype=dtype, device="cuda")
    desc = eg.make_attn_desc(1, 1, d, dtype)
    out = torch.full_like(q, float("nan"))
    eg.engram_attn_paged(desc, q, cu_of([1] * seqs), cache.kv_len, cache.table, cache.k, cache.v, out, max_q)
    assert eg.engram_check_errors() == 0
    for i in range(0, seqs, 13):
        ref = reference(q[i:i + 1], cache.keys[i], cache.values[i], scale)
        assert ref[0].min() > 0.005       # there is a tail to lose
        assert_tail_close(out[i:i + 1], ref, dtype, d, scale)


def test_a_long_tail_in_a_prompt():
    # the same for the last rows of prompts; each has one sharp key, and 150 prompts fill the CTAs
    n, seqs, d, dtype = 700, 150, 64, F16
    scale = 1 / math.sqrt(d)
    k = torch.zeros((seqs, n, 1, d), dtype=dtype, device="cuda")
    k[:, 0] = 25.6 * math.log(2) / scale / d
    v = (torch.rand((seqs, n, 1, d), device="cuda") * 1024 + 512).to(dtype)
    v[:, 0] = 0
    q = torch.ones_like(k)
    k, v, q = (t.view(seqs * n, 1, d) for t in (k, v, q))
    out = torch.full_like(q, float("nan"))
    eg.engram_attn_prompt(eg.make_attn_desc(1, 1, d, dtype), q, k, v, cu_of([n] * seqs), out)
    assert eg.engram_check_errors() == 0
    for i in range(0, seqs, 29):
        s = slice(i * n, (i + 1) * n)
        ref = reference(q[s], k[s], v[s], scale)
        assert ref[0][-1].min() > 0.005
        assert_tail_close(out[s], ref, dtype, d, scale)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("max_q", [1, 64], ids=["few rows", "tiles"])
def test_scores_far_apart_keep_their_sums(max_q, dtype):
    # maxima that rise by small and large steps from tile to tile: what is rescaled, and the largest
    # probabilities against a maximum that lags, stay in the type's range
    lens, d, heads = [1999, 640, 3, 1100], 128, 2
    cache = Paged(lens, 16, 1, d, dtype, 33)
    for i, n in enumerate(lens):
        rise = torch.linspace(0, (40.0, 6.0, 3.0, -30.0)[i], n, device="cuda")
        k = (rise * math.sqrt(d) / d)[:, None, None].expand(n, 1, d) + 0.02 * randn((n, 1, d), 50 + i, torch.float32)
        cache.keys[i] = k.to(dtype)
        cache.write(i, 0, cache.keys[i], cache.values[i])
    q = (torch.ones((4, heads, d), device="cuda") + 0.1 * randn((4, heads, d), 60, torch.float32)).to(dtype)
    out, lse = torch.full_like(q, float("nan")), torch.zeros((4, heads), device="cuda")
    desc, scale = eg.make_attn_desc(heads, 1, d, dtype), 1 / math.sqrt(d)
    eg.engram_attn_paged(desc, q, cu_of([1] * 4), cache.kv_len, cache.table, cache.k, cache.v, out, max_q, lse_out=lse)
    assert eg.engram_check_errors() == 0
    for i in range(4):
        ref = reference(q[i:i + 1], cache.keys[i], cache.values[i], scale)
        assert_tail_close(out[i:i + 1], ref, dtype, d, scale)
        assert (np.abs(f64(lse[i:i + 1]) - ref[1]) <= tolerance(ref, dtype, d, scale)[1]).all()
