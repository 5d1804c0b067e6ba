"""Serving over a paged key-value cache: append new tokens, attend with one new token per sequence,
and evict what has drawn the least attention.

    paged_append(k, v, k_cache, v_cache, page_table, seq_lens, ...)
    out = paged_attn(q, k_cache, v_cache, page_table, seq_lens + 1, max_seq_len, ...)
    seq_lens = paged_evict(k_cache, v_cache, mass, key_positions, page_table, seq_lens, budget, ...)

The cache is the caller's: ``k_cache`` / ``v_cache`` [num_pages, Hkv, page_size, d] (HND) or
[num_pages, page_size, Hkv, d] (NHD) in fp16 or bf16, ``page_table`` int32 [B, max_pages], ``seq_lens``
int32 [B]. Token slot t of sequence b lies in page ``page_table[b, t // page_size]`` at
``t % page_size``. Eviction keeps two planes beside it, ``mass`` (float32) and ``key_positions`` (int32),
both [num_pages, Hkv, page_size]. Lengths and pages are read on the device, so a step can be
captured into a CUDA graph; ``read_device_status(workspace)`` tells of bad ones.
"""

import contextlib
import ctypes

import torch

from . import DTYPE, LAYOUT, _check, _check_workspace, _lib, _packed, _stream_ptr, alloc_workspace
from ._lib import SagePagedCache

__all__ = ["paged_attn", "paged_append", "paged_evict", "paged_attn_workspace_bytes",
           "paged_evict_workspace_bytes"]

STATUS_BYTES = 256


def _on(stream):
    """Allocations made for a call on another stream belong to that stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _check_small(name, t, shape, dtype, device):
    if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} {list(shape)} tensor on the inputs' device")


def _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions):
    """Shapes, types and devices of a cache; returns (num_pages, heads_kv, page_size, head_dim)."""
    if tensor_layout not in LAYOUT:
        raise ValueError("tensor_layout must be 'HND' or 'NHD'")
    if k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must be 4-D and of one shape")
    if k_cache.dtype not in DTYPE or v_cache.dtype != k_cache.dtype:
        raise TypeError("k_cache and v_cache must share one dtype, float16 or bfloat16")
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("page_table and seq_lens must be int32")
    if page_table.dim() != 2 or (page_table.numel() and page_table.stride(1) != 1):
        raise ValueError("page_table must be [batch, max_pages] with contiguous rows")
    if seq_lens.dim() != 1 or seq_lens.shape[0] != page_table.shape[0] or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous [batch] tensor")
    if tensor_layout == "HND":
        pages, heads, size, d = k_cache.shape
    else:
        pages, size, heads, d = k_cache.shape
    dev = k_cache.device
    _check_small("mass", mass, (pages, heads, size), torch.float32, dev)
    _check_small("key_positions", key_positions, (pages, heads, size), torch.int32, dev)
    if not all(t.device == dev for t in (v_cache, page_table, seq_lens)):
        raise ValueError("the cache, its page table and seq_lens must be on one device")
    return pages, heads, size, d


def _check_cuda(dev, workspace):
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    _check_workspace(workspace, dev)


def _cache(k_cache, v_cache, page_table, seq_lens, size, mass, key_positions):
    for t in (k_cache, v_cache):
        if t.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
    return SagePagedCache(k_cache.data_ptr(), (ctypes.c_int64 * 3)(*k_cache.stride()[:3]), v_cache.data_ptr(),
                          (ctypes.c_int64 * 3)(*v_cache.stride()[:3]), k_cache.shape[0], size,
                          page_table.data_ptr(), page_table.stride(0), page_table.shape[1], seq_lens.data_ptr(),
                          0 if mass is None else mass.data_ptr(),
                          0 if key_positions is None else key_positions.data_ptr())


def paged_attn_workspace_bytes(batch, heads_q, heads_kv, max_seq_len, head_dim, accumulate=False):
    return _lib.load().sage_paged_attn_workspace_size(batch, heads_q, heads_kv, max_seq_len, head_dim,
                                                      int(bool(accumulate)))


def paged_evict_workspace_bytes(batch, heads_kv, max_seq_len, budget):
    return _lib.load().sage_paged_evict_workspace_size(batch, heads_kv, max_seq_len, budget)


def paged_attn(q, k_cache, v_cache, page_table, seq_lens, max_seq_len, tensor_layout="HND", sm_scale=None,
               softcap=0.0, slopes=None, key_positions=None, q_positions=None, mass=None, return_lse=False,
               out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [B, Hq, d], over the ``seq_lens`` tokens its cache holds
    (its own key and value included). Returns out (q's shape and dtype), plus lse [B, Hq] fp32 if
    return_lse; a sequence that holds nothing gives 0 and -inf.

    ``max_seq_len``: an upper bound of seq_lens. ``softcap`` > 0: scores become
    softcap·tanh(s / softcap). ``slopes`` fp32 [Hq]: slopes[h]·|q_position - key position| is taken off;
    the key's position is its slot unless ``key_positions`` gives it (a cache that was evicted from), the
    query's is seq_len - 1 unless ``q_positions`` int32 [B] does. ``mass``: the weight each held token
    draws, summed over the query heads of its key/value head, is added to it in place."""
    pages, hkv, size, d = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions)
    if q.dim() != 3 or q.shape[0] != page_table.shape[0] or q.shape[2] != d:
        raise ValueError("q must be [batch, heads, head_dim] with the cache's batch and head_dim")
    if q.dtype != k_cache.dtype:
        raise TypeError("q must have the cache's dtype")
    if q.device != k_cache.device:
        raise ValueError("q must be on the cache's device")
    B, hq, _ = q.shape
    dev = q.device
    if out is not None and (tuple(out.shape) != tuple(q.shape) or out.dtype != q.dtype or out.device != dev):
        raise ValueError("out must have q's shape, dtype and device")
    _check_small("slopes", slopes, (hq,), torch.float32, dev)
    _check_small("q_positions", q_positions, (B,), torch.int32, dev)
    if return_lse:
        _check_small("lse", lse, (B, hq), torch.float32, dev)
    _check_cuda(dev, workspace)
    lib = _lib.load()
    with torch.cuda.device(dev), _on(stream):
        if out is None:
            out = torch.empty((B, hq, d), dtype=q.dtype, device=dev)
        if return_lse and lse is None:
            lse = torch.empty((B, hq), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = alloc_workspace(lib.sage_paged_attn_workspace_size(
                B, hq, hkv, int(max_seq_len), d, int(mass is not None)), dev)
        cache = _cache(k_cache, v_cache, page_table, seq_lens, size, mass, key_positions)
        st = lib.sage_paged_attn(ctypes.byref(_packed(q)), ctypes.byref(cache), ctypes.byref(_packed(out)),
                                 _ptr(lse if return_lse else None), _ptr(slopes), _ptr(q_positions), B, hq, hkv,
                                 int(max_seq_len), d, DTYPE[q.dtype], LAYOUT[tensor_layout],
                                 float("nan") if sm_scale is None else float(sm_scale), float(softcap),
                                 _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(st, "paged_attn")
    return (out, lse) if return_lse else out


def paged_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, tensor_layout="HND", mass=None,
                 key_positions=None, positions=None, workspace=None, stream=None):
    """Writes new tokens k, v [T, Hkv, d] behind the ``seq_lens`` tokens their sequences hold (seq_lens is
    not raised). ``cu_seqlens`` int32 [B + 1] says which tokens are whose; without it each sequence gets
    one. Tokens behind the last sequence are left out. ``mass`` becomes 0 in the new slots,
    ``key_positions`` the token's entry of ``positions`` int32 [T], or its slot. A token whose slot or page
    is not in the cache is left out, and recorded in ``workspace`` (256 bytes) where one is given."""
    pages, hkv, size, d = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions)
    if k.dim() != 3 or tuple(v.shape) != tuple(k.shape) or tuple(k.shape[1:]) != (hkv, d):
        raise ValueError("k and v must be [tokens, heads, head_dim] with the cache's heads and head_dim")
    if k.dtype != k_cache.dtype or v.dtype != k.dtype:
        raise TypeError("k and v must have the cache's dtype")
    if k.device != k_cache.device or v.device != k.device:
        raise ValueError("k and v must be on the cache's device")
    B, T, dev = page_table.shape[0], k.shape[0], k.device
    if cu_seqlens is None and T != B:
        raise ValueError("without cu_seqlens every sequence gets one token")
    _check_small("cu_seqlens", cu_seqlens, (B + 1,), torch.int32, dev)
    _check_small("positions", positions, (T,), torch.int32, dev)
    if positions is not None and key_positions is None:
        raise ValueError("positions need the key_positions plane")
    _check_cuda(dev, workspace)
    lib = _lib.load()
    with torch.cuda.device(dev):
        cache = _cache(k_cache, v_cache, page_table, seq_lens, size, mass, key_positions)
        st = lib.sage_paged_append(ctypes.byref(_packed(k)), ctypes.byref(_packed(v)), ctypes.byref(cache),
                                   _ptr(cu_seqlens), _ptr(positions), B, T, hkv, d, DTYPE[k.dtype],
                                   LAYOUT[tensor_layout], _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream_ptr(stream))
    _check(st, "paged_append")


def paged_evict(k_cache, v_cache, mass, key_positions, page_table, seq_lens, budget, max_seq_len, sink=0, recent=0,
                tensor_layout="HND", workspace=None, stream=None):
    """Cuts every sequence that holds more than ``budget`` tokens down to ``budget``, in place, and returns the
    new lengths int32 [B]. For each key/value head, tokens at positions below ``sink`` or among the last
    ``recent`` positions stay, then those with the largest ``mass`` (ties: the lowest slot). Kept tokens
    behind the budget move into the freed slots, with their mass and position; the slots behind the
    budget keep what they held, and their pages are free."""
    pages, hkv, size, d = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions)
    if mass is None or key_positions is None:
        raise ValueError("eviction needs the mass and key_positions planes")
    if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError("budget must be at least 1 and hold sink + recent tokens")
    B, dev = page_table.shape[0], k_cache.device
    _check_cuda(dev, workspace)
    lib = _lib.load()
    with torch.cuda.device(dev), _on(stream):
        new_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = alloc_workspace(lib.sage_paged_evict_workspace_size(B, hkv, int(max_seq_len), int(budget)), dev)
        cache = _cache(k_cache, v_cache, page_table, seq_lens, size, mass, key_positions)
        st = lib.sage_paged_evict(ctypes.byref(cache), _ptr(new_lens), B, hkv, int(max_seq_len), d,
                                  DTYPE[k_cache.dtype], LAYOUT[tensor_layout], int(budget), int(sink), int(recent),
                                  _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(st, "paged_evict")
    return new_lens
