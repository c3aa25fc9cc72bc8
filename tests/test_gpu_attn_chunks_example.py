"""GPU: the serving example with chunks of several tokens after the prompt (a prompt's second part,
drafted tokens): every step's attention is that of the oracle over all positions so far."""
import numpy as np
import pytest
import torch

import synth
from examples.serve_layer import Layer, dev
from oracle.attention import attend
from tests.attn_helpers import assert_attn_close, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [[20, 5, 1, 3], [1, 4, 30], [40, 40]])
def test_chunks_after_the_prompt(steps):
    geom, batch, heads, kv_heads, head_dim = synth.TINY, 2, 4, 2, 64
    layer = Layer(geom, heads, kv_heads, head_dim, batch, sum(steps), 16, 3)
    scale = head_dim ** -0.5
    keys, values = [[] for _ in range(batch)], [[] for _ in range(batch)]
    for i, n in enumerate(steps):
        b = synth.make_batch(geom, batch, n, 20 + i)
        _, q, k, v, out = layer.step(dev(b.x).view(torch.bfloat16), dev(b.tokens))
        for j in range(batch):
            s = slice(j * n, (j + 1) * n)
            keys[j].append(f64(k[s]))
            values[j].append(f64(v[s]))
            ref = attend(f64(q[s]), np.concatenate(keys[j]), np.concatenate(values[j]), scale)
            assert_attn_close(out[s], None, ref, torch.bfloat16, head_dim, scale)
    assert layer.length.tolist() == [sum(steps)] * batch
