"""Page tables of a paged cache kept on the GPU: sequences that grow take pages from a stack of free ones,
sequences that shrink or end give theirs back.

    free_pages = torch.arange(num_pages, dtype=torch.int32, device=dev)     # the stack: its first free_count entries
    free_count = torch.tensor([num_pages], dtype=torch.int32, device=dev)
    a = paged_assign(page_table, seq_lens, add_lens, free_pages, free_count, page_size, max_tokens)
    paged_append(k, v, k_cache, v_cache, page_table, a.held_lens, cu_seqlens=a.cu_seqlens)
    seq_lens, free_count = a.seq_lens, a.free_count
    ...
    free_count = paged_release(page_table, seq_lens, keep_lens, free_pages, free_count, page_size)
    seq_lens = keep_lens

A page belongs to one sequence: one that two sequences hold would come back twice. Nothing is read back by the host, so a
step can be captured into a CUDA graph.
"""

import functools
from typing import NamedTuple

import torch

from . import SageError, _check_workspace, _lib
from .paged import _check_range, _check_small, _Launch, _ptr, _Scratch

__all__ = ["PageAssignment", "paged_assign", "paged_release", "paged_release_workspace_bytes"]


class PageAssignment(NamedTuple):
    """What ``paged_assign`` returns, all on the device."""
    seq_lens: torch.Tensor    # int32 [B]: lengths with the new tokens; as before where a sequence was not served
    held_lens: torch.Tensor   # int32 [B]: lengths before, -1 where not served: the appends' seq_lens
    cu_seqlens: torch.Tensor  # int32 [B + 1]: where each sequence's new tokens lie in packed rows
    positions: torch.Tensor   # int32 [max_tokens]: the new tokens' positions, -1 behind the last
    slots: torch.Tensor       # int64 [max_tokens]: page · page_size + place of each new token, -1 where it has none
    free_count: torch.Tensor  # int32 [1]: pages left on the stack


def _check_table(page_table, free_pages, free_count, page_size, workspace):
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError("page_table must be an int32 [batch, max_pages] tensor with contiguous rows")
    index = page_table.get_device()
    _check_small("free_pages", free_pages, (free_pages.numel(),), torch.int32, index)
    _check_small("free_count", free_count, (1,), torch.int32, index)
    if page_size < 1:
        raise ValueError("page_size must be at least 1")
    _check_range("page_size", page_size)
    if workspace is not None:
        _check_workspace(workspace, page_table.device)
    return page_table.shape[0], page_table.shape[1], index


def paged_assign(page_table, seq_lens, add_lens, free_pages, free_count, page_size, max_tokens, next_positions=None,
                 workspace=None, stream=None):
    """Pages for ``add_lens`` int32 [B] new tokens of sequences that hold ``seq_lens`` int32 [B]. In their order, sequences
    take the pages they lack from the top of the stack (the first ``free_count`` int32 [1] entries of ``free_pages`` int32
    [num_pages], which is not changed) into their rows of ``page_table``, in place; once one finds too few, it and all
    later ones that need pages take none. Returns a ``PageAssignment``.

    ``max_tokens``: an upper bound of the new tokens, the size of the maps. ``next_positions`` int32 [B]: the position of
    each sequence's first new token, where a sequence that was evicted from counts on; default: seq_lens. A sequence whose
    lengths are negative, do not fit its row of the table, or whose tokens end behind max_tokens is not served;
    ``read_device_status(workspace)`` tells of it where a workspace (256 bytes) is given, as of a count out of range."""
    B, width, index = _check_table(page_table, free_pages, free_count, page_size, workspace)
    _check_small("seq_lens", seq_lens, (B,), torch.int32, index)
    _check_small("add_lens", add_lens, (B,), torch.int32, index)
    if next_positions is not None:
        _check_small("next_positions", next_positions, (B,), torch.int32, index)
    n = _check_range("max_tokens", max_tokens)
    if index < 0:
        raise ValueError("the page table must be on a CUDA device")
    with _Launch(index, stream) as on:
        dev = page_table.device
        # (tensors of their own: views of one cost the host 4 us more)
        lens, held, count = torch.empty_like(seq_lens), torch.empty_like(seq_lens), torch.empty_like(free_count)
        cu = torch.empty((B + 1,), dtype=torch.int32, device=dev)
        positions = torch.empty((n,), dtype=torch.int32, device=dev)
        slots = torch.empty((n,), dtype=torch.int64, device=dev)
        st = _lib.load().sage_paged_assign(page_table.data_ptr(), page_table.stride(0), width, _ptr(seq_lens), _ptr(add_lens),
                                           _ptr(next_positions), _ptr(free_pages), _ptr(free_count), free_pages.numel(),
                                           page_size, B, n, _ptr(lens), _ptr(held), _ptr(cu), _ptr(positions), _ptr(slots),
                                           _ptr(count), _ptr(workspace), 0 if workspace is None else workspace.numel(), on)
    if st:
        raise SageError(st, "paged_assign")
    return PageAssignment(lens, held, cu, positions, slots, count)


@functools.lru_cache(1024)
def paged_release_workspace_bytes(batch):
    return _lib.load().sage_paged_release_workspace_size(batch)


def paged_release(page_table, seq_lens, keep_lens, free_pages, free_count, page_size, workspace=None, stream=None):
    """Gives back the pages behind the first ``keep_lens`` int32 [B] of the ``seq_lens`` int32 [B] tokens that sequences hold:
    after an eviction (keep_lens the new lengths), or of ended sequences (0). The pages go onto the stack, ``free_pages`` from
    ``free_count`` on, in place and in the order of the sequences and their rows; returns the new count int32 [1]. The
    page table is not changed. A sequence with bad lengths or pages gives nothing, and where the stack has no room that
    sequence and the later ones do not (``read_device_status``)."""
    B, width, index = _check_table(page_table, free_pages, free_count, page_size, workspace)
    _check_small("seq_lens", seq_lens, (B,), torch.int32, index)
    _check_small("keep_lens", keep_lens, (B,), torch.int32, index)
    if index < 0:
        raise ValueError("the page table must be on a CUDA device")
    lib = _lib.load()
    with _Launch(index, stream) as on:
        count = torch.empty((1,), dtype=torch.int32, device=page_table.device)
        # (more than a status word: the pages that each sequence gives)
        with _Scratch(workspace, paged_release_workspace_bytes(B) + 1, on) as w:
            st = lib.sage_paged_release(page_table.data_ptr(), page_table.stride(0), width, _ptr(seq_lens), _ptr(keep_lens),
                                        _ptr(free_pages), _ptr(free_count), free_pages.numel(), page_size, B, _ptr(count),
                                        w.at, w.nbytes, on)
    if st:
        raise SageError(st, "paged_release")
    return count
