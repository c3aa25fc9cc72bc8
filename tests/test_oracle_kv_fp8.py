"""Pins of the 8-bit cache's oracle (no GPU): the scale is the smallest that fits, a code is the nearest one,
what fits exactly comes back as it was, and torch's own types agree."""
import numpy as np
import torch

from oracle import kv_fp8
from oracle.numerics import e4m3_to_f64


def test_scale_is_the_smallest_that_fits():
    tops = np.array([448.0, 448.0 * (1 + 2.0 ** -20), 224.0, 224.1, 1.0, 2.0 ** -10, 1.75, 1.7500001, 3.3e38, 2.0 ** -92])
    x = np.zeros((len(tops), 16))
    x[:, 3] = -tops
    _, s = kv_fp8.quantise(x)
    f = np.ldexp(1.0, s.astype(int) - 127)
    assert (tops <= 448 * f).all()
    assert (tops[:-1] > 448 * f[:-1] / 2).all() and s[-1] == 27      # no smaller scale than 2^-100
    np.testing.assert_array_equal(s[:4].astype(int) - 127, [0, 1, -1, 0])


def test_zeros_and_not_finite():
    x = np.zeros((4, 16))
    x[0, 1] = -0.0
    x[1, 2], x[2, 3], x[3, :] = np.inf, np.nan, 2.0 ** -130
    c, s = kv_fp8.quantise(x)
    assert s.tolist() == [127, 255, 255, 27]
    assert c[0].tolist() == [0, 0x80] + [0] * 14 and not c[1:].any()
    v = kv_fp8.values(c, s)
    assert (v[0] == 0).all() and np.isnan(v[1:3]).all() and (v[3] == 0).all()


def test_codes_are_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((300, 48)) * np.exp2(rng.integers(-60, 60, (300, 1)))
    c, s = kv_fp8.quantise(x)
    v = kv_fp8.values(c, s)
    every = np.sort(e4m3_to_f64(np.array([i for i in range(256) if i & 127 != 127], dtype=np.uint8)))
    f = np.ldexp(1.0, s.astype(int) - 127)[:, None]
    near = np.abs(x[..., None] / f[..., None] - every).min(-1)
    np.testing.assert_array_equal(np.abs(x - v), near * f)
    assert (np.abs(x - v) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * f)).all()
    # a second time, nothing changes
    c2, s2 = kv_fp8.quantise(v)
    np.testing.assert_array_equal(kv_fp8.values(c2, s2), v)


def test_torch_agrees():
    x = torch.randn((50, 32), dtype=torch.float64)
    c, s = kv_fp8.quantise(x.numpy())
    f = torch.from_numpy(s).view(torch.float8_e8m0fnu).double()[:, None]
    want = (x / f).float().to(torch.float8_e4m3fn)
    assert torch.equal(want.view(torch.uint8), torch.from_numpy(c))
    np.testing.assert_array_equal((want.double() * f).numpy(), kv_fp8.values(c, s))
    assert kv_fp8.values(np.array([[0x38]]), np.array([0]))[0, 0] == 2.0 ** -100     # below 27 counts as 27
