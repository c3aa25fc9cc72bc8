"""GPU: the serving example. The block and the attention run together on one length array; the
attention's outputs of the prompt and of every decoding step are those of the float64 oracle over
the queries, keys and values that went in."""
import numpy as np
import pytest
import torch

from examples.serve_layer import serve
from oracle.attention import attend
from tests.attn_helpers import assert_attn_close, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prompt,steps,heads,kv_heads,head_dim,page", [
    (3, 40, 4, 8, 2, 64, 16), (2, 200, 3, 6, 2, 128, 24), (5, 2, 6, 4, 4, 80, 8)])
def test_serving_matches_the_oracle(batch, prompt, steps, heads, kv_heads, head_dim, page):
    layer, got = serve(batch, prompt, steps, heads, kv_heads, head_dim, page)
    assert layer.length.tolist() == [prompt + steps] * batch
    scale = head_dim ** -0.5
    for b in range(batch):
        keys, values = [], []
        for i, (streams, q, k, v, out) in enumerate(got):
            n = prompt if i == 0 else 1
            assert torch.isfinite(streams.float()).all()
            s = slice(b * n, (b + 1) * n)
            keys.append(f64(k[s]))
            values.append(f64(v[s]))
            ref = attend(f64(q[s]), np.concatenate(keys), np.concatenate(values), scale)
            assert_attn_close(out[s], None, ref, torch.bfloat16, head_dim, scale)
