"""GPU: the serving example with its attention's cache in eight bits: the prompt's attention is that over the
keys and values in hand, every later step's that over the quantised ones, which read back as the oracle has
them."""
import numpy as np
import pytest
import torch

from examples.serve_layer import serve
from oracle import kv_fp8
from oracle.attention import attend
from oracle.numerics import e4m3_to_f64
from tests.attn_helpers import assert_attn_close, f64
from tests.fp8_helpers import PagedFp8, assert_close, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prompt,steps,heads,kv_heads,head_dim,page", [
    (3, 40, 4, 8, 2, 64, 16), (2, 200, 3, 6, 2, 128, 48), (5, 2, 6, 4, 4, 80, 16)])
def test_serving_matches_the_oracle(batch, prompt, steps, heads, kv_heads, head_dim, page):
    layer, got = serve(batch, prompt, steps, heads, kv_heads, head_dim, page, eight_bits=True)
    assert layer.length.tolist() == [prompt + steps] * batch
    scale, total = head_dim ** -0.5, prompt + steps
    read = [f64(x).reshape(batch, total, kv_heads, head_dim) for x in layer.cached(total)]
    for b in range(batch):
        cache = PagedFp8.__new__(PagedFp8)
        parts = {n: [] for n in ("keys", "values", "codes", "exponents")}
        for i, (streams, q, k, v, out) in enumerate(got):
            n = prompt if i == 0 else 1
            assert torch.isfinite(streams.float()).all()
            s = slice(b * n, (b + 1) * n)
            kc, ks = kv_fp8.quantise(f64(k[s]))
            vc, vs = kv_fp8.quantise(f64(v[s]))
            for name, x in (("keys", kv_fp8.values(kc, ks)), ("values", kv_fp8.values(vc, vs)),
                            ("codes", e4m3_to_f64(vc)), ("exponents", vs.astype(np.int64) - 127)):
                parts[name].append(x)
                setattr(cache, name, [np.concatenate(parts[name])])
            if i == 0:
                ref = attend(f64(q[s]), f64(k[s]), f64(v[s]), scale)
                assert_attn_close(out[s], None, ref, torch.bfloat16, head_dim, scale)
            else:
                assert_close(out[s], None, *reference(cache, 0, q[s], scale), torch.bfloat16, head_dim, scale,
                             heads // kv_heads)
        np.testing.assert_array_equal(read[0][b], cache.keys[0])
        np.testing.assert_array_equal(read[1][b], cache.values[0])
