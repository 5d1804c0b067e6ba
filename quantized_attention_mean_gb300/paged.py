"""Serving over a paged key-value cache: append new tokens, attend with one new token per sequence,
and evict what has drawn the least attention.

    paged_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens, mass=mass, key_positions=positions)
    seq_lens = seq_lens + prompt_lens   # the calls read the lengths, the caller raises them
    next_pos = seq_lens.clone()         # the next token's position: from the first eviction on not its slot
    for q_new, k_new, v_new in steps:   # one token of every sequence at a time
        paged_append(k_new, v_new, k_cache, v_cache, page_table, seq_lens, mass=mass, key_positions=positions,
                     positions=next_pos)
        seq_lens = seq_lens + 1
        out = paged_attn(q_new, k_cache, v_cache, page_table, seq_lens, max_len, softcap=50.0, slopes=slopes,
                         key_positions=positions, q_positions=next_pos, mass=mass)
        seq_lens = paged_evict(k_cache, v_cache, mass, positions, page_table, seq_lens, budget, max_len, sink=4, recent=128)
        next_pos = next_pos + 1

The cache is the caller's: ``k_cache`` / ``v_cache`` [num_pages, Hkv, page_size, d] (HND) or
[num_pages, page_size, Hkv, d] (NHD) in fp16 or bf16, ``page_table`` int32 [B, max_pages], ``seq_lens``
int32 [B]. Token slot t of sequence b lies in page ``page_table[b, t // page_size]`` at
``t % page_size``. Eviction keeps two planes beside it, ``mass`` (float32) and ``key_positions`` (int32),
both [num_pages, Hkv, page_size]. Lengths and pages are read on the device, so a step can be
captured into a CUDA graph; ``read_device_status(workspace)`` tells of bad ones.
"""

import contextlib
import functools
from ctypes import byref

import torch

from . import DTYPE, LAYOUT, SageError, _check_workspace, _lib
from ._lib import SagePacked, SagePagedCache

__all__ = ["paged_attn", "paged_append", "paged_evict", "paged_attn_workspace_bytes",
           "paged_evict_workspace_bytes"]

STATUS_BYTES = 256
INT32_MAX = 2 ** 31 - 1
_NAN = float("nan")  # sm_scale: the default


class _Launch:
    """The device and stream a call runs on; what it allocates belongs to that stream. (A decode step is a few
    microseconds of GPU time, so the ordinary case, the current device and stream, enters no context.)"""

    __slots__ = ("contexts", "stream")

    def __init__(self, index, stream):
        self.contexts = None
        if stream is not None or torch._C._cuda_getDevice() != index:
            with contextlib.ExitStack() as stack:
                stack.enter_context(torch.cuda.device(index))
                if stream is not None:
                    stack.enter_context(torch.cuda.stream(stream))
                self.contexts = stack.pop_all()
        self.stream = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        if self.contexts is not None:
            self.contexts.close()


def _ptr(t):
    return None if t is None else t.data_ptr()


class _Scratch:
    """A call's workspace: the caller's, or memory of PyTorch's allocator that belongs to the launching stream and
    goes back to it after the launch (straight from the allocator: a tensor costs the host 2 us more). None for
    a status word alone, which no one could read."""

    __slots__ = ("at", "nbytes", "mine")

    def __init__(self, workspace, nbytes, stream):
        self.mine = False
        if workspace is not None:
            self.at, self.nbytes = workspace.data_ptr(), workspace.numel()
        elif nbytes <= STATUS_BYTES:
            self.at, self.nbytes = None, 0
        else:
            self.at, self.nbytes = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, stream), nbytes
            self.mine = True

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self.mine:
            torch._C._cuda_cudaCachingAllocator_raw_delete(self.at)


def _check_small(name, t, shape, dtype, index):
    if t is not None and (t.dtype != dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} {list(shape)} tensor on the inputs' device")


def _check_range(name, value):
    """Sizes go to the library as 32-bit integers, which would wrap silently."""
    if not 0 <= value <= INT32_MAX:
        raise ValueError(f"{name} must be in [0, 2^31)")
    return int(value)


def _packed(t):
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.shape[2] != 1:
        raise ValueError("the last dimension must be contiguous")
    return SagePacked(t.data_ptr(), s0, s1)


def _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions, workspace):
    """Shapes, types and devices of a cache; returns its description and (heads_kv, head_dim, device index)."""
    if tensor_layout not in LAYOUT:
        raise ValueError("tensor_layout must be 'HND' or 'NHD'")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be 4-D and of one shape")
    if k_cache.dtype not in DTYPE or v_cache.dtype != k_cache.dtype:
        raise TypeError("k_cache and v_cache must share one dtype, float16 or bfloat16")
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("page_table and seq_lens must be int32")
    if page_table.dim() != 2 or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError("page_table must be [batch, max_pages] with contiguous rows")
    batch, width = page_table.shape
    if seq_lens.dim() != 1 or seq_lens.shape[0] != batch or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous [batch] tensor")
    if tensor_layout == "HND":
        pages, heads, size, d = shape
    else:
        pages, size, heads, d = shape
    index = k_cache.get_device()
    if mass is not None:
        _check_small("mass", mass, (pages, heads, size), torch.float32, index)
    if key_positions is not None:
        _check_small("key_positions", key_positions, (pages, heads, size), torch.int32, index)
    if v_cache.get_device() != index or page_table.get_device() != index or seq_lens.get_device() != index:
        raise ValueError("the cache, its page table and seq_lens must be on one device")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if d != 1 and (k3 != 1 or v3 != 1):
        raise ValueError("the last dimension must be contiguous")
    if workspace is not None:
        _check_workspace(workspace, k_cache.device)
    cache = SagePagedCache(k_cache.data_ptr(), k0, k1, k2, v_cache.data_ptr(), v0, v1, v2, pages, size,
                           page_table.data_ptr(), page_table.stride(0), width, seq_lens.data_ptr(), _ptr(mass),
                           _ptr(key_positions))
    return cache, heads, d, index


def _check_cuda(index):
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")


@functools.lru_cache(1024)
def paged_attn_workspace_bytes(batch, heads_q, heads_kv, max_seq_len, head_dim, accumulate=False):
    return _lib.load().sage_paged_attn_workspace_size(batch, heads_q, heads_kv, max_seq_len, head_dim,
                                                      int(bool(accumulate)))


@functools.lru_cache(1024)
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
    query's is seq_len - 1 unless ``q_positions`` int32 [B] does. Once a sequence has been evicted from, its slots and its
    length are no positions any more: with ``slopes`` give both. ``mass``: the weight each held token
    draws, summed over the query heads of its key/value head, is added to it in place; it takes a workspace of
    4·B·Hq·max_seq_len bytes, whatever the lengths. A sequence whose length lies outside of [0, max_seq_len] or of the
    table counts as empty, a token whose page is not in the cache as a row of zeros; ``read_device_status(workspace)``
    tells of either, and nothing does where no workspace is given."""
    cache, hkv, d, index = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions,
                                        workspace)
    shape = q.shape
    if len(shape) != 3 or shape[0] != page_table.shape[0] or shape[2] != d:
        raise ValueError("q must be [batch, heads, head_dim] with the cache's batch and head_dim")
    if q.dtype != k_cache.dtype:
        raise TypeError("q must have the cache's dtype")
    if q.get_device() != index:
        raise ValueError("q must be on the cache's device")
    B, hq, _ = shape
    if out is not None and (out.shape != shape or out.dtype != q.dtype or out.get_device() != index):
        raise ValueError("out must have q's shape, dtype and device")
    if slopes is not None:
        _check_small("slopes", slopes, (hq,), torch.float32, index)
    if q_positions is not None:
        _check_small("q_positions", q_positions, (B,), torch.int32, index)
    if not return_lse:
        lse = None
    elif lse is not None:
        _check_small("lse", lse, (B, hq), torch.float32, index)
    _check_cuda(index)
    n = _check_range("max_seq_len", max_seq_len)
    lib = _lib.load()
    with _Launch(index, stream) as on:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        if return_lse and lse is None:
            lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
        nbytes = 0 if workspace is not None else paged_attn_workspace_bytes(B, hq, hkv, n, d, mass is not None)
        with _Scratch(workspace, nbytes, on) as w:
            st = lib.sage_paged_attn(byref(_packed(q)), byref(cache), byref(_packed(out)), _ptr(lse), _ptr(slopes),
                                     _ptr(q_positions), B, hq, hkv, n, d, DTYPE[q.dtype], LAYOUT[tensor_layout],
                                     _NAN if sm_scale is None else sm_scale, softcap, w.at, w.nbytes, on)
    if st:
        raise SageError(st, "paged_attn")
    return (out, lse) if return_lse else out


def paged_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, tensor_layout="HND", mass=None,
                 key_positions=None, positions=None, workspace=None, stream=None):
    """Writes new tokens k, v [T, Hkv, d] behind the ``seq_lens`` tokens their sequences hold (seq_lens is
    not raised). ``cu_seqlens`` int32 [B + 1] says which tokens are whose; without it each sequence gets
    one. Tokens behind the last sequence are left out. ``mass`` becomes 0 in the new slots,
    ``key_positions`` the token's entry of ``positions`` int32 [T], or its slot. A token whose slot or page
    is not in the cache is left out, as are all of a sequence of negative length, and recorded in
    ``workspace`` (256 bytes) where one is given. Once a sequence has been evicted from, ``key_positions`` needs
    ``positions``: a new token's slot then lies below the positions that were kept, and the next eviction would
    take it for an old one."""
    cache, hkv, d, index = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions,
                                        workspace)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != hkv or shape[2] != d:
        raise ValueError("k and v must be [tokens, heads, head_dim] with the cache's heads and head_dim")
    if k.dtype != k_cache.dtype or v.dtype != k.dtype:
        raise TypeError("k and v must have the cache's dtype")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError("k and v must be on the cache's device")
    B, T = page_table.shape[0], shape[0]
    if cu_seqlens is None:
        if T != B:
            raise ValueError("without cu_seqlens every sequence gets one token")
    else:
        _check_small("cu_seqlens", cu_seqlens, (B + 1,), torch.int32, index)
    if positions is not None:
        _check_small("positions", positions, (T,), torch.int32, index)
        if key_positions is None:
            raise ValueError("positions need the key_positions plane")
    _check_cuda(index)
    _check_range("the number of tokens", T)
    with _Launch(index, stream) as on:
        st = _lib.load().sage_paged_append(byref(_packed(k)), byref(_packed(v)), byref(cache), _ptr(cu_seqlens),
                                           _ptr(positions), B, T, hkv, d, DTYPE[k.dtype], LAYOUT[tensor_layout],
                                           _ptr(workspace), 0 if workspace is None else workspace.numel(), on)
    if st:
        raise SageError(st, "paged_append")


def paged_evict(k_cache, v_cache, mass, key_positions, page_table, seq_lens, budget, max_seq_len, sink=0, recent=0,
                tensor_layout="HND", workspace=None, stream=None):
    """Cuts every sequence that holds more than ``budget`` tokens down to ``budget``, in place, and returns the
    new lengths int32 [B]. For each key/value head, tokens at positions below ``sink`` or among the last
    ``recent`` positions stay, then those with the largest ``mass`` (ties: the lowest slot). Kept tokens
    behind the budget move into the freed slots, with their mass and position; the slots behind the
    budget keep what they held, and their pages are free. Positions that count on from the kept ones make new tokens
    the last ones: give ``positions`` to ``paged_append`` from then on. Only ``paged_attn`` adds mass: right after a prompt
    every mass is 0, and besides the protected tokens the lowest slots stay. A sequence with a bad length or page is left as it was, its
    length too (``read_device_status``)."""
    if mass is None or key_positions is None:
        raise ValueError("eviction needs the mass and key_positions planes")
    cache, hkv, d, index = _check_cache(k_cache, v_cache, page_table, seq_lens, tensor_layout, mass, key_positions,
                                        workspace)
    if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError("budget must be at least 1 and hold sink + recent tokens")
    B = page_table.shape[0]
    _check_cuda(index)
    n, budget = _check_range("max_seq_len", max_seq_len), _check_range("budget", budget)
    lib = _lib.load()
    with _Launch(index, stream) as on:
        new_lens = torch.empty((B,), dtype=torch.int32, device=k_cache.device)
        nbytes = 0 if workspace is not None else paged_evict_workspace_bytes(B, hkv, n, budget)
        with _Scratch(workspace, nbytes, on) as w:
            st = lib.sage_paged_evict(byref(cache), new_lens.data_ptr(), B, hkv, n, d, DTYPE[k_cache.dtype],
                                      LAYOUT[tensor_layout], budget, sink, recent, w.at, w.nbytes, on)
    if st:
        raise SageError(st, "paged_evict")
    return new_lens
