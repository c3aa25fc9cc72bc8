"""Host check that the block's binding refuses tensors and streams of another device than the one that
the library launches on (no GPU: tensors that only say where they are)."""
import types

import pytest
import torch

from deepseek_v4_engram_gb300 import api


class On(torch.Tensor):
    """A CPU tensor that says it is on a CUDA device."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def on(at):
    t = torch.zeros(4, dtype=torch.int32).as_subclass(On)
    t.at = at
    return t


def test_tensors_and_streams_have_to_be_on_the_current_device(monkeypatch):
    monkeypatch.setattr(api, "_current_device", lambda: 0, raising=False)
    t = on(0)
    assert api._ptr(t, "i32", "tokens") == t.data_ptr()
    with pytest.raises(ValueError, match="tokens: on cuda:1"):
        api._ptr(on(1), "i32", "tokens")
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        api._ptr(torch.zeros(4, dtype=torch.int32), "i32", "tokens")
    assert api._stream(types.SimpleNamespace(cuda_stream=77, device_index=0)).value == 77
    with pytest.raises(ValueError, match="stream: on cuda:1"):
        api._stream(types.SimpleNamespace(cuda_stream=77, device_index=1))
