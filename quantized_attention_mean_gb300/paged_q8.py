"""Serving over a paged key-value cache held in 8 bits, with a scale for each block of tokens and head.

    k_cache = torch.zeros(num_pages, Hkv, page_size, d, dtype=torch.int8)            # HND; NHD as in the 16-bit calls
    v_cache = torch.zeros(num_pages, Hkv, page_size, d, dtype=torch.float8_e4m3fn)   # either type for either cache
    k_scales = torch.zeros(num_pages, Hkv, page_size // block)                       # float32, block divides page_size
    q, k = qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight)
    paged_append_q8(k, v, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, cu_seqlens)
    seq_lens = seq_lens + prompt_lens        # the calls read the lengths, the caller raises them
    out = paged_attn_q8(q_new, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, max_len)

Token slot t of sequence b lies in page ``page_table[b, t // page_size]`` at ``t % page_size``; its scale is that of block
``t % page_size // block`` of the page and head, its value code · scale. Scales follow the tokens: the largest magnitude in
a block decides, and a token that needs a larger scale than its block has makes the block's codes be rounded again. Keys are
rounded as they are: what all keys have in common in a channel, which ``sage_attn`` takes off first, widens their scale (int8
keys of unit variance about channel means of size 4: results off by 6% instead of 2%; E4M3 keys four times as much). A cache
in 8 bits has no mass or position planes: it is not evicted from (``paged_evict`` takes 16-bit caches).
"""

import functools
from ctypes import byref

import torch

from . import DTYPE, LAYOUT, SageError, _check_workspace, _lib
from ._lib import SageQ8Cache
from .paged import (_NAN, _check_cuda, _check_range, _check_small, _Launch, _packed, _ptr, _Scratch)

__all__ = ["paged_attn_q8", "paged_append_q8", "paged_read_q8", "paged_attn_q8_workspace_bytes"]

CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}


def _check_q8(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, tensor_layout, workspace):
    """Shapes, types and devices of an 8-bit cache; returns its description and (heads_kv, head_dim, device index)."""
    if tensor_layout not in LAYOUT:
        raise ValueError("tensor_layout must be 'HND' or 'NHD'")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be 4-D and of one shape")
    if k_cache.dtype not in CODES or v_cache.dtype not in CODES:
        raise TypeError("k_cache and v_cache must be int8 or float8_e4m3fn")
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
    blocks = k_scales.shape[2] if k_scales.dim() == 3 else 0
    if blocks < 1 or size % blocks:
        raise ValueError("k_scales must be [num_pages, heads, page_size / block] with a block that divides page_size")
    _check_small("k_scales", k_scales, (pages, heads, blocks), torch.float32, index)
    _check_small("v_scales", v_scales, (pages, heads, blocks), torch.float32, index)
    if v_cache.get_device() != index or page_table.get_device() != index or seq_lens.get_device() != index:
        raise ValueError("the cache, its page table and seq_lens must be on one device")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if d != 1 and (k3 != 1 or v3 != 1):
        raise ValueError("the last dimension must be contiguous")
    if workspace is not None:
        _check_workspace(workspace, k_cache.device)
    cache = SageQ8Cache(k_cache.data_ptr(), k0, k1, k2, v_cache.data_ptr(), v0, v1, v2, k_scales.data_ptr(),
                        v_scales.data_ptr(), CODES[k_cache.dtype], CODES[v_cache.dtype], pages, size, size // blocks,
                        page_table.data_ptr(), page_table.stride(0), width, seq_lens.data_ptr())
    return cache, heads, d, index


@functools.lru_cache(1024)
def paged_attn_q8_workspace_bytes(batch, heads_q, heads_kv, max_seq_len, head_dim):
    return _lib.load().sage_paged_attn_q8_workspace_size(batch, heads_q, heads_kv, max_seq_len, head_dim)


def paged_attn_q8(q, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, max_seq_len, tensor_layout="HND",
                  sm_scale=None, softcap=0.0, slopes=None, q_positions=None, return_lse=False, out=None, lse=None,
                  workspace=None, stream=None):
    """``paged_attn`` over an 8-bit cache: attention of one new token per sequence, q [B, Hq, d] in fp16 or bf16, over the
    ``seq_lens`` tokens its cache holds (its own key and value included). Returns out (q's shape and dtype), plus lse
    [B, Hq] fp32 if return_lse; a sequence that holds nothing gives 0 and -inf. A key's position, for ``slopes``, is its
    slot. Scales must be finite and not negative; slots and scales behind the held tokens may hold anything. A sequence
    whose length lies outside of [0, max_seq_len] or of the table counts as empty, a token whose page is not in the cache as
    a row of zeros; ``read_device_status(workspace)`` tells of either, and nothing does where no workspace is given."""
    cache, hkv, d, index = _check_q8(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, tensor_layout, workspace)
    shape = q.shape
    if len(shape) != 3 or shape[0] != page_table.shape[0] or shape[2] != d:
        raise ValueError("q must be [batch, heads, head_dim] with the cache's batch and head_dim")
    if q.dtype not in DTYPE:
        raise TypeError("q must be float16 or bfloat16")
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
        nbytes = 0 if workspace is not None else paged_attn_q8_workspace_bytes(B, hq, hkv, n, d)
        with _Scratch(workspace, nbytes, on) as w:
            st = lib.sage_paged_attn_q8(byref(_packed(q)), byref(cache), byref(_packed(out)), _ptr(lse), _ptr(slopes),
                                        _ptr(q_positions), B, hq, hkv, n, d, DTYPE[q.dtype], LAYOUT[tensor_layout],
                                        _NAN if sm_scale is None else sm_scale, softcap, w.at, w.nbytes, on)
    if st:
        raise SageError(st, "paged_attn_q8")
    return (out, lse) if return_lse else out


def _check_new(name, k, v, hkv, d, index):
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != hkv or shape[2] != d:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with the cache's heads and head_dim")
    if k.dtype not in DTYPE or v.dtype != k.dtype:
        raise TypeError(f"{name} must share one dtype, float16 or bfloat16")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError(f"{name} must be on the cache's device")
    return _check_range("the number of tokens", shape[0])


def paged_append_q8(k, v, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, cu_seqlens=None,
                    tensor_layout="HND", workspace=None, stream=None):
    """``paged_append`` into an 8-bit cache: writes new tokens k, v [T, Hkv, d] (fp16 or bf16, finite) as codes behind the
    ``seq_lens`` tokens their sequences hold (seq_lens is not raised). ``cu_seqlens`` int32 [B + 1] says which tokens are
    whose; without it each sequence gets one. Tokens behind the last sequence are left out, and so are those before the first
    (``cu_seqlens[0]`` should be 0), those whose slot or page is not in the cache and all of a sequence of negative length (these
    are recorded in ``workspace``, 256 bytes, where given).

    The scale of a block becomes ``max(s, need, 2^-100)``: s that of its earlier tokens, 0 if the first new token begins the
    block; need = max|x| / 127 for int8, the smallest power of two with max|x| ≤ 448 · need for E4M3. Codes are x / scale
    rounded to nearest even; where the scale grew, the earlier codes are multiplied by old / new and rounded again, which
    for E4M3 loses nothing but bits of the smallest values. Two sequences must not append to one block, nor one sequence
    to a block whose page others read."""
    cache, hkv, d, index = _check_q8(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, tensor_layout, workspace)
    T = _check_new("k and v", k, v, hkv, d, index)
    B = page_table.shape[0]
    if cu_seqlens is None:
        if T != B:
            raise ValueError("without cu_seqlens every sequence gets one token")
    else:
        _check_small("cu_seqlens", cu_seqlens, (B + 1,), torch.int32, index)
    _check_cuda(index)
    with _Launch(index, stream) as on:
        st = _lib.load().sage_paged_append_q8(byref(_packed(k)), byref(_packed(v)), byref(cache), _ptr(cu_seqlens), B, T,
                                              hkv, d, DTYPE[k.dtype], LAYOUT[tensor_layout], _ptr(workspace),
                                              0 if workspace is None else workspace.numel(), on)
    if st:
        raise SageError(st, "paged_append_q8")


def paged_read_q8(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, cu_seqlens, tokens, starts=None,
                  dtype=torch.bfloat16, tensor_layout="HND", k_out=None, v_out=None, workspace=None, stream=None):
    """Values of held tokens as packed rows k, v [tokens, Hkv, d] in ``dtype`` (fp16 or bf16; new tensors unless k_out and
    v_out are given): what the next chunk of a prompt attends to with ``scored_attn``. Rows ``cu_seqlens[b]`` up to
    ``cu_seqlens[b + 1]`` (int32 [B + 1]) are the slots from ``starts[b]`` on (int32 [B], default 0) of sequence b. Rows of no
    held token become 0: behind seq_lens or of a bad page (``read_device_status``), or behind the last sequence."""
    cache, hkv, d, index = _check_q8(k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, tensor_layout, workspace)
    T, B = _check_range("tokens", tokens), page_table.shape[0]
    if dtype not in DTYPE:
        raise TypeError("dtype must be float16 or bfloat16")
    _check_small("cu_seqlens", cu_seqlens, (B + 1,), torch.int32, index)
    if starts is not None:
        _check_small("starts", starts, (B,), torch.int32, index)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and (t.shape != (T, hkv, d) or t.dtype != dtype or t.get_device() != index):
            raise ValueError(f"{name} must be a {str(dtype)[6:]} [{T}, {hkv}, {d}] tensor on the cache's device")
    _check_cuda(index)
    with _Launch(index, stream) as on:
        if k_out is None:
            k_out = torch.empty((T, hkv, d), dtype=dtype, device=k_cache.device)
        if v_out is None:
            v_out = torch.empty((T, hkv, d), dtype=dtype, device=k_cache.device)
        st = _lib.load().sage_paged_read_q8(byref(_packed(k_out)), byref(_packed(v_out)), byref(cache), _ptr(cu_seqlens),
                                            _ptr(starts), B, T, hkv, d, DTYPE[dtype], LAYOUT[tensor_layout], _ptr(workspace),
                                            0 if workspace is None else workspace.numel(), on)
    if st:
        raise SageError(st, "paged_read_q8")
    return k_out, v_out
