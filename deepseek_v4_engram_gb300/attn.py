"""Binding of the attention operators of libengram.so: the entry points of include/engram.h under
the same names. Argument checks and marshalling only, as in api.py.

Queries, keys, values and outputs are CUDA tensors [tokens, heads, head_dim] of torch.bfloat16 or
torch.float16 whose last dimension is dense (views of a wider buffer are fine). A paged cache is a
pair of tensors [pages, page_size, kv_heads, head_dim] with a block table int32 [sequences, width].
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import EngramAttnDesc, EngramAttnView, EngramKvCache
from .api import _check, _stream, lib

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
_TORCH = {_lib.BF16: torch.bfloat16, _lib.F16: torch.float16}


def make_attn_desc(n_heads: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                   scale: float | None = None) -> EngramAttnDesc:
    """`scale` multiplies the products of queries and keys (default head_dim^-1/2)."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype: expected torch.bfloat16 or torch.float16, got {dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    return EngramAttnDesc(n_heads, n_kv_heads, head_dim, _DTYPES[dtype], scale)


def _tensor(t, name: str, ndim: int, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the library takes device pointers)")
    if t.dtype != dtype or t.dim() != ndim:
        raise ValueError(f"{name}: expected a {ndim}-dimensional {dtype} tensor, got "
                         f"{t.dim()}-dimensional {t.dtype}")


def _view(t, name: str, heads: int, desc: EngramAttnDesc, tokens: int | None = None):
    _tensor(t, name, 3, _TORCH[desc.dtype])
    n, h, d = t.shape
    if h != heads or d != desc.head_dim or (tokens is not None and n != tokens):
        want = "tokens" if tokens is None else tokens
        raise ValueError(f"{name}: expected shape [{want}, {heads}, {desc.head_dim}], got "
                         f"{[n, h, d]}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return EngramAttnView(t.data_ptr(), s[0], s[1])


def _ints(t, name: str, count: int | None = None):
    _tensor(t, name, 1, torch.int32)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if count is not None and t.shape[0] != count:
        raise ValueError(f"{name}: expected {count} elements, got {t.shape[0]}")
    return t.data_ptr()


def _sequences(cu_seqlens) -> int:
    n = cu_seqlens.shape[0] - 1 if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() else 0
    if n < 0:
        raise ValueError("cu_seqlens: expected one element more than there are sequences")
    return n


def _cache(desc: EngramAttnDesc, k_cache, v_cache, block_table, n_seqs: int):
    dtype = _TORCH[desc.dtype]
    _tensor(k_cache, "k_cache", 4, dtype)
    _tensor(v_cache, "v_cache", 4, dtype)
    _tensor(block_table, "block_table", 2, torch.int32)
    pages, page_size, heads, d = k_cache.shape
    if heads != desc.n_kv_heads or d != desc.head_dim or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache: expected [pages, page_size, {desc.n_kv_heads}, "
                         f"{desc.head_dim}], got {list(k_cache.shape)} and {list(v_cache.shape)}")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache and v_cache: the last dimension must be dense")
    if block_table.shape[0] != n_seqs or not block_table.is_contiguous():
        raise ValueError(f"block_table: expected a contiguous [{n_seqs}, width] tensor")
    return EngramKvCache(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1],
                         vs[2], pages, page_size, block_table.data_ptr(), block_table.shape[1])


def _scratch(desc: EngramAttnDesc, workspace, device):
    """The given workspace, or a fresh one."""
    if workspace is None:
        workspace = torch.empty(engram_attn_workspace_size(desc), dtype=torch.uint8, device=device)
    else:
        _tensor(workspace, "workspace", 1, torch.uint8)
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
    return workspace


def _lse(lse_out, tokens: int, desc: EngramAttnDesc):
    if lse_out is None:
        return None
    _tensor(lse_out, "lse_out", 2, torch.float32)
    if lse_out.shape != (tokens, desc.n_heads) or not lse_out.is_contiguous():
        raise ValueError(f"lse_out: expected a contiguous [{tokens}, {desc.n_heads}] tensor")
    return lse_out.data_ptr()


def engram_attn_workspace_size(desc: EngramAttnDesc) -> int:
    return int(lib().engram_attn_workspace_size(ctypes.byref(desc)))


def engram_attn_prompt(desc: EngramAttnDesc, q, k, v, cu_seqlens, out, workspace=None,
                       lse_out=None, stream=None):
    """Causal attention over the packed sequences cu_seqlens (int32 [sequences + 1]) of q, k and
    v. `workspace` (uint8, engram_attn_workspace_size bytes) defaults to a fresh one."""
    qv = _view(q, "q", desc.n_heads, desc)
    total = q.shape[0]
    kv = _view(k, "k", desc.n_kv_heads, desc, total)
    vv = _view(v, "v", desc.n_kv_heads, desc, total)
    ov = _view(out, "out", desc.n_heads, desc, total)
    workspace = _scratch(desc, workspace, q.device)
    _check(lib().engram_attn_prompt(
        ctypes.byref(desc), ctypes.byref(qv), ctypes.byref(kv), ctypes.byref(vv),
        _ints(cu_seqlens, "cu_seqlens"), _sequences(cu_seqlens), total, ctypes.byref(ov),
        _lse(lse_out, total, desc), workspace.data_ptr(), workspace.numel(), _stream(stream)))


def engram_attn_paged(desc: EngramAttnDesc, q, cu_seqlens, kv_len, block_table, k_cache, v_cache,
                      out, max_q: int, workspace=None, lse_out=None, stream=None):
    """Attention of the chunks cu_seqlens of q over the caches: kv_len (int32 [sequences]) counts
    the chunks' own positions. `max_q` is the longest chunk."""
    qv = _view(q, "q", desc.n_heads, desc)
    total = q.shape[0]
    ov = _view(out, "out", desc.n_heads, desc, total)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, k_cache, v_cache, block_table, n)
    workspace = _scratch(desc, workspace, q.device)
    _check(lib().engram_attn_paged(
        ctypes.byref(desc), ctypes.byref(qv), _ints(cu_seqlens, "cu_seqlens"), n, total, max_q,
        _ints(kv_len, "kv_len", n), ctypes.byref(cache), ctypes.byref(ov),
        _lse(lse_out, total, desc), workspace.data_ptr(), workspace.numel(), _stream(stream)))


def engram_kv_append(desc: EngramAttnDesc, k, v, cu_seqlens, kv_len, block_table, k_cache, v_cache,
                     stream=None):
    """Write the chunks' keys and values into the caches' pages; kv_len already counts them."""
    kv = _view(k, "k", desc.n_kv_heads, desc)
    total = k.shape[0]
    vv = _view(v, "v", desc.n_kv_heads, desc, total)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, k_cache, v_cache, block_table, n)
    _check(lib().engram_kv_append(
        ctypes.byref(desc), ctypes.byref(kv), ctypes.byref(vv), _ints(cu_seqlens, "cu_seqlens"),
        n, total, _ints(kv_len, "kv_len", n), ctypes.byref(cache), _stream(stream)))
