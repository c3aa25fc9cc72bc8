"""Host check that the attention binding refuses tensors and streams of another device than the one that
the library launches on (no GPU: tensors that only say where they are, and a library that counts calls)."""
import types

import pytest
import torch

from deepseek_v4_engram_gb300 import attn


class On(torch.Tensor):
    """A CPU tensor that says it is on a CUDA device."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def on(shape, dtype, at=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.at = at
    return t


@pytest.fixture
def calls(monkeypatch):
    made = []

    def entry(name):
        return lambda *a: made.append((name, a[-1])) or 0
    names = ("engram_attn_prompt", "engram_attn_paged", "engram_kv_append")
    fake = types.SimpleNamespace(engram_attn_workspace_size=lambda d: 64, **{n: entry(n) for n in names})
    monkeypatch.setattr(attn, "lib", lambda: fake)
    monkeypatch.setattr(attn, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(attn, "_raw_stream", lambda device: 1000 + device)
    return made


DESC = attn.make_attn_desc(4, 2, 64)
BF16 = torch.bfloat16


def arguments(name):
    heads = {"q": 4, "out": 4, "k": 2, "v": 2}
    a = {n: on((5, h, 64), BF16) for n, h in heads.items()}
    a["cu_seqlens"], a["kv_len"] = on(3, torch.int32), on(2, torch.int32)
    a["block_table"] = on((2, 4), torch.int32)
    a["k_cache"], a["v_cache"] = (on((8, 16, 2, 64), BF16) for _ in range(2))
    a["workspace"], a["lse_out"] = on(64, torch.uint8), on((5, 4), torch.float32)
    keep = {"engram_attn_prompt": "q k v cu_seqlens out workspace lse_out",
            "engram_attn_paged": "q cu_seqlens kv_len block_table k_cache v_cache out workspace lse_out",
            "engram_kv_append": "k v cu_seqlens kv_len block_table k_cache v_cache"}[name].split()
    a = {n: a[n] for n in keep}
    if name == "engram_attn_paged":
        a["max_q"] = 3
    return a


@pytest.mark.parametrize("name", ["engram_attn_prompt", "engram_attn_paged", "engram_kv_append"])
def test_every_tensor_has_to_be_on_the_current_device(calls, name):
    call, a = getattr(attn, name), arguments(name)
    call(DESC, **a)
    stream = types.SimpleNamespace(cuda_stream=77, device_index=0)
    call(DESC, stream=stream, **a)
    assert calls == [(name, 1000), (name, 77)]
    for n, t in a.items():
        if not isinstance(t, On):
            continue
        moved = on(t.shape, t.dtype, 1)
        with pytest.raises(ValueError, match="cuda:1"):
            call(DESC, **dict(a, **{n: moved}))
        with pytest.raises(ValueError):          # and a CPU tensor
            call(DESC, **dict(a, **{n: torch.zeros(t.shape, dtype=t.dtype)}))
    # all of them on a device that is not the current one
    with pytest.raises(ValueError, match="current device"):
        call(DESC, **{n: on(t.shape, t.dtype, 1) if isinstance(t, On) else t for n, t in a.items()})
    with pytest.raises(ValueError, match="stream"):
        call(DESC, stream=types.SimpleNamespace(cuda_stream=77, device_index=1), **a)
    assert len(calls) == 2
