"""Binding of the attention operators of libengram.so: the entry points of include/engram.h under
the same names. Argument checks and marshalling only, as in api.py.

Queries, keys, values and outputs are CUDA tensors [tokens, heads, head_dim] of torch.bfloat16 or
torch.float16 whose last dimension is dense (views of a wider buffer are fine). A paged cache is a
pair of tensors [pages, page_size, kv_heads, head_dim] with a block table int32 [sequences, width].
The library launches on the thread's current device, so every tensor of a call has to be there.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import EngramAttnDesc
from .api import _check, lib

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
_TORCH = {_lib.BF16: torch.bfloat16, _lib.F16: torch.float16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_pack_view, _pack_cache = _lib.PACK_VIEW.pack, _lib.PACK_CACHE.pack


def make_attn_desc(n_heads: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                   scale: float | None = None) -> EngramAttnDesc:
    """`scale` multiplies the products of queries and keys (default head_dim^-1/2)."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype: expected torch.bfloat16 or torch.float16, got {dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    return EngramAttnDesc(n_heads, n_kv_heads, head_dim, _DTYPES[dtype], scale)


# A decoding step's calls are shorter on the GPU than a chain of careful helpers on the host, so
# each check below is one expression of cheap tensor attributes; what is wrong with an argument
# that fails it is worked out only then. Views and caches go to the library as packed bytes, which take
# a quarter of the time of filling a ctypes Structure and a reference to it.

def _refuse(t, name: str, shape: str, dtype, device: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the library takes device pointers)")
    if t.get_device() != device:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the call's device is cuda:{device}")
    raise ValueError(f"{name}: expected a {dtype} tensor {shape}, got {t.dtype} {list(t.shape)} "
                     f"with strides {t.stride()}")


def _device(t, name: str, stream) -> int:
    """The device of a call: the current one, which its first tensor and its stream must be on."""
    device = t.get_device() if isinstance(t, torch.Tensor) else -1
    if device < 0:
        _refuse(t, name, "", None, device)
    if device != _current_device():
        raise ValueError(f"{name}: on cuda:{device}, but the current device, where the library "
                         f"launches, is cuda:{_current_device()}")
    if stream is not None and stream.device_index != device:
        raise ValueError(f"stream: on cuda:{stream.device_index}, the call's device is cuda:{device}")
    return device


def _view(t, name: str, heads: int, dim: int, dtype, device: int, tokens: int = -1):
    if isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype:
        shape = t.shape
        if len(shape) == 3 and shape[1] == heads and shape[2] == dim and (
                tokens < 0 or shape[0] == tokens):
            s = t.stride()
            if s[2] == 1:
                return _pack_view(t.data_ptr(), s[0], s[1])
    n = "tokens" if tokens < 0 else tokens
    _refuse(t, name, f"[{n}, {heads}, {dim}] whose last dimension is dense", dtype, device)


def _ints(t, name: str, device: int, count: int = -1):
    if isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is torch.int32:
        shape = t.shape
        if len(shape) == 1 and (count < 0 or shape[0] == count) and t.is_contiguous():
            return t.data_ptr()
    _refuse(t, name, f"[{'n' if count < 0 else count}], contiguous", torch.int32, device)


def _sequences(cu_seqlens) -> int:
    n = cu_seqlens.shape[0] - 1
    if n < 0:
        raise ValueError("cu_seqlens: expected one element more than there are sequences")
    return n


def _cache(desc: EngramAttnDesc, dtype, k_cache, v_cache, block_table, device: int, n_seqs: int):
    if (isinstance(k_cache, torch.Tensor) and isinstance(v_cache, torch.Tensor)
            and isinstance(block_table, torch.Tensor) and k_cache.get_device() == device
            and v_cache.get_device() == device and block_table.get_device() == device
            and k_cache.dtype is dtype and v_cache.dtype is dtype
            and block_table.dtype is torch.int32):
        shape, table = k_cache.shape, block_table.shape
        if (len(shape) == 4 and shape[2] == desc.n_kv_heads and shape[3] == desc.head_dim
                and v_cache.shape == shape and len(table) == 2 and table[0] == n_seqs
                and block_table.is_contiguous()):
            k0, k1, k2, k3 = k_cache.stride()
            v0, v1, v2, v3 = v_cache.stride()
            if k3 == 1 and v3 == 1:
                return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2,
                                   shape[0], shape[1], block_table.data_ptr(), table[1])
    want = (f"[pages, page_size, {desc.n_kv_heads}, {desc.head_dim}] whose last dimension is "
            f"dense, keys and values alike, with a contiguous int32 block_table [{n_seqs}, width]")
    for t in (k_cache, v_cache, block_table):
        if not isinstance(t, torch.Tensor) or t.get_device() != device:
            _refuse(t, "k_cache, v_cache and block_table", want, dtype, device)
    _refuse(k_cache, "k_cache, v_cache and block_table", want, dtype, device)


def _scratch(desc: EngramAttnDesc, workspace, device: int, stream):
    """The given workspace, or a fresh one. That belongs to the call's stream: the allocator may hand
    its memory on as soon as the call returns, to the next user in the order of that stream."""
    if workspace is None:
        if stream is not None:
            with torch.cuda.stream(stream):
                return _scratch(desc, None, device, None)
        return torch.empty(engram_attn_workspace_size(desc), dtype=torch.uint8, device=device)
    if not (isinstance(workspace, torch.Tensor) and workspace.get_device() == device
            and workspace.dtype is torch.uint8 and workspace.is_contiguous()):
        _refuse(workspace, "workspace", "[bytes], contiguous", torch.uint8, device)
    return workspace


def _lse(lse_out, tokens: int, desc: EngramAttnDesc, device: int):
    if lse_out is None:
        return None
    if not (isinstance(lse_out, torch.Tensor) and lse_out.get_device() == device
            and lse_out.dtype is torch.float32 and lse_out.shape == (tokens, desc.n_heads)
            and lse_out.is_contiguous()):
        _refuse(lse_out, "lse_out", f"[{tokens}, {desc.n_heads}], contiguous", torch.float32,
                device)
    return lse_out.data_ptr()


def _stream(stream, device: int):
    """The given stream, or the device's current one."""
    return _raw_stream(device) if stream is None else stream.cuda_stream


def engram_attn_workspace_size(desc: EngramAttnDesc) -> int:
    return int(lib().engram_attn_workspace_size(ctypes.byref(desc)))


def engram_attn_prompt(desc: EngramAttnDesc, q, k, v, cu_seqlens, out, workspace=None,
                       lse_out=None, stream=None):
    """Causal attention over the packed sequences cu_seqlens (int32 [sequences + 1]) of q, k and
    v. `workspace` (uint8, engram_attn_workspace_size bytes) defaults to a fresh one."""
    dtype, heads, kv_heads, dim = _TORCH[desc.dtype], desc.n_heads, desc.n_kv_heads, desc.head_dim
    device = _device(q, "q", stream)
    qv = _view(q, "q", heads, dim, dtype, device)
    total = q.shape[0]
    kv = _view(k, "k", kv_heads, dim, dtype, device, total)
    vv = _view(v, "v", kv_heads, dim, dtype, device, total)
    ov = _view(out, "out", heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    workspace = _scratch(desc, workspace, device, stream)
    _check(lib().engram_attn_prompt(
        ctypes.byref(desc), qv, kv, vv, cu, _sequences(cu_seqlens), total, ov,
        _lse(lse_out, total, desc, device),
        workspace.data_ptr(), workspace.numel(), _stream(stream, device)))


def engram_attn_paged(desc: EngramAttnDesc, q, cu_seqlens, kv_len, block_table, k_cache, v_cache,
                      out, max_q: int, workspace=None, lse_out=None, stream=None):
    """Attention of the chunks cu_seqlens of q over the caches: kv_len (int32 [sequences]) counts
    the chunks' own positions. `max_q` is the longest chunk; it picks the kernel."""
    dtype, heads, dim = _TORCH[desc.dtype], desc.n_heads, desc.head_dim
    device = _device(q, "q", stream)
    qv = _view(q, "q", heads, dim, dtype, device)
    total = q.shape[0]
    ov = _view(out, "out", heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, dtype, k_cache, v_cache, block_table, device, n)
    workspace = _scratch(desc, workspace, device, stream)
    _check(lib().engram_attn_paged(
        ctypes.byref(desc), qv, cu, n, total, max_q, _ints(kv_len, "kv_len", device, n),
        cache, ov, _lse(lse_out, total, desc, device), workspace.data_ptr(),
        workspace.numel(), _stream(stream, device)))


def engram_kv_append(desc: EngramAttnDesc, k, v, cu_seqlens, kv_len, block_table, k_cache, v_cache,
                     stream=None):
    """Write the chunks' keys and values into the caches' pages; kv_len already counts them."""
    dtype, kv_heads, dim = _TORCH[desc.dtype], desc.n_kv_heads, desc.head_dim
    device = _device(k, "k", stream)
    kv = _view(k, "k", kv_heads, dim, dtype, device)
    total = k.shape[0]
    vv = _view(v, "v", kv_heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, dtype, k_cache, v_cache, block_table, device, n)
    _check(lib().engram_kv_append(
        ctypes.byref(desc), kv, vv, cu, n, total,
        _ints(kv_len, "kv_len", device, n), cache, _stream(stream, device)))
