"""Binding of the operators on an 8-bit cache of libengram.so: the entry points of include/engram.h
under the same names. Argument checks and marshalling only, as in attn.py.

A paged cache is four tensors: the codes of keys and values, torch.float8_e4m3fn (or the same bits as
torch.uint8) [pages, page_size, kv_heads, head_dim] whose last dimension is dense, and their scales,
torch.float8_e8m0fnu (or torch.uint8) [pages, kv_heads, page_size] whose last dimension is dense, with a
block table int32 [sequences, width]. One scale belongs to a position and key-value head.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import EngramAttnDesc
from .api import _check, lib
from .attn import _TORCH, _device, _ints, _lse, _refuse, _scratch, _sequences, _stream, _view

_U8, _CODES, _INT = torch.uint8, torch.float8_e4m3fn, torch.int32
_SCALES = getattr(torch, "float8_e8m0fnu", None)   # an older torch has no such type: scales are uint8 there
_pack_cache = _lib.PACK_CACHE_FP8.pack


def _cache(desc: EngramAttnDesc, k_cache, v_cache, k_scale, v_scale, block_table, device: int, n_seqs: int):
    try:   # what is no tensor, or has another number of dimensions, ends here
        pages, page_size, heads, dim = shape = k_cache.shape
        k0, k1, k2, k3 = k_cache.stride()
        v0, v1, v2, v3 = v_cache.stride()
        a0, a1, a2 = k_scale.stride()
        b0, b1, b2 = v_scale.stride()
        n, width = block_table.shape
        codes, scales, of_scales = k_cache.dtype, k_scale.dtype, k_scale.shape
        if (k_cache.get_device() == device and v_cache.get_device() == device and k_scale.get_device() == device
                and v_scale.get_device() == device and block_table.get_device() == device
                and (codes is _U8 or codes is _CODES) and v_cache.dtype is codes
                and (scales is _U8 or scales is _SCALES) and v_scale.dtype is scales and block_table.dtype is _INT
                and heads == desc.n_kv_heads and dim == desc.head_dim and n == n_seqs and v_cache.shape == shape
                and of_scales == (pages, heads, page_size) and v_scale.shape == of_scales
                and k3 == 1 and v3 == 1 and a2 == 1 and b2 == 1 and block_table.is_contiguous()):
            return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                               k0, k1, k2, v0, v1, v2, a0, a1, b0, b1, pages, page_size, block_table.data_ptr(), width)
    except (AttributeError, TypeError, ValueError):
        pass
    name = "k_cache, v_cache, k_scale, v_scale and block_table"
    want = (f"[pages, page_size, {desc.n_kv_heads}, {desc.head_dim}] whose last dimension is dense, keys and values "
            f"alike, with scales [pages, {desc.n_kv_heads}, page_size] whose last dimension is dense and a contiguous "
            f"int32 block_table [{n_seqs}, width]")
    for t in (k_cache, v_cache, k_scale, v_scale, block_table):
        if not isinstance(t, torch.Tensor) or t.get_device() != device:
            _refuse(t, name, want, "float8_e4m3fn or uint8", device)
    for t, of in ((v_cache, k_cache), (v_scale, k_scale)):   # the one to name: keys, unless the values differ
        if t.dtype is not of.dtype or t.shape != of.shape:
            _refuse(t, name, want, "float8_e4m3fn or uint8", device)
    _refuse(k_cache, name, want, "float8_e4m3fn or uint8", device)


def engram_kv_append_fp8(desc: EngramAttnDesc, k, v, cu_seqlens, kv_len, block_table, k_cache, v_cache, k_scale,
                         v_scale, stream=None):
    """Quantise the chunks' keys and values into the caches' pages; kv_len already counts them."""
    dtype, kv_heads, dim = _TORCH[desc.dtype], desc.n_kv_heads, desc.head_dim
    device = _device(k, "k", stream)
    kv = _view(k, "k", kv_heads, dim, dtype, device)
    total = k.shape[0]
    vv = _view(v, "v", kv_heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, k_cache, v_cache, k_scale, v_scale, block_table, device, n)
    _check(lib().engram_kv_append_fp8(ctypes.byref(desc), kv, vv, cu, n, total, _ints(kv_len, "kv_len", device, n),
                                      cache, _stream(stream, device)))


def engram_kv_read_fp8(desc: EngramAttnDesc, cu_seqlens, kv_len, block_table, k_cache, v_cache, k_scale, v_scale,
                       k_out, v_out, stream=None):
    """Read the chunks' keys and values (the last positions of each sequence, or all of them) back into
    k_out and v_out [tokens, kv_heads, head_dim] of the descriptor's type."""
    dtype, kv_heads, dim = _TORCH[desc.dtype], desc.n_kv_heads, desc.head_dim
    device = _device(k_out, "k_out", stream)
    kv = _view(k_out, "k_out", kv_heads, dim, dtype, device)
    total = k_out.shape[0]
    vv = _view(v_out, "v_out", kv_heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, k_cache, v_cache, k_scale, v_scale, block_table, device, n)
    _check(lib().engram_kv_read_fp8(ctypes.byref(desc), cu, n, total, _ints(kv_len, "kv_len", device, n), cache, kv,
                                    vv, _stream(stream, device)))


def engram_attn_paged_fp8(desc: EngramAttnDesc, q, cu_seqlens, kv_len, block_table, k_cache, v_cache, k_scale,
                          v_scale, out, max_q: int, workspace=None, lse_out=None, stream=None):
    """Attention of the chunks cu_seqlens of q over the caches: kv_len (int32 [sequences]) counts the chunks' own
    positions. `max_q` is the longest chunk; it picks the kernel. `workspace` as for engram_attn_paged."""
    dtype, heads, dim = _TORCH[desc.dtype], desc.n_heads, desc.head_dim
    device = _device(q, "q", stream)
    qv = _view(q, "q", heads, dim, dtype, device)
    total = q.shape[0]
    ov = _view(out, "out", heads, dim, dtype, device, total)
    cu = _ints(cu_seqlens, "cu_seqlens", device)
    n = _sequences(cu_seqlens)
    cache = _cache(desc, k_cache, v_cache, k_scale, v_scale, block_table, device, n)
    workspace = _scratch(desc, workspace, device, stream)
    _check(lib().engram_attn_paged_fp8(
        ctypes.byref(desc), qv, cu, n, total, max_q, _ints(kv_len, "kv_len", device, n), cache, ov,
        _lse(lse_out, total, desc, device), workspace.data_ptr(), workspace.numel(), _stream(stream, device)))
