"""Attention with modified scores: capped by a tanh, biased by distance, under document and prefix
masks, on 16-bit operands. For the layers whose scores the quantised calls cannot take."""

import functools
from ctypes import byref

import torch

from . import DTYPE, LAYOUT, SageError, _check_dense_args, _dims, _lib
from ._lib import SageView
from .paged import _NAN, _check_small, _Launch, _ptr, _Scratch

__all__ = ["scored_attn", "scored_attn_workspace_bytes"]


def _view(t, whole):
    """t for the library, and whether the kernel can read its rows in place (`whole`: head_dim is a multiple
    of 8; otherwise, and where an address or stride is not, rows are copied to the workspace)."""
    n0, n1, n2, n3 = t.shape
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and n3 != 1:
        raise ValueError("the last dimension must be contiguous")
    at = t.data_ptr()
    return SageView(at, s0, s1, s2), (whole and at % 16 == 0 and (n0 <= 1 or (s0 > 0 and s0 % 8 == 0))
                                      and (n1 <= 1 or (s1 > 0 and s1 % 8 == 0))
                                      and (n2 <= 1 or (s2 > 0 and s2 % 8 == 0)))


@functools.lru_cache(1024)
def scored_attn_workspace_bytes(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim, packed=True, documents=True):
    """``packed``: q, k and v have 16-byte aligned rows (address, strides and head_dim). ``documents``: doc_ids are given."""
    return _lib.load().sage_scored_attn_workspace_size(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim,
                                                       int(bool(packed)) + 2 * (not documents))


def scored_attn(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None, softcap=0.0, slopes=None,
                prefix_lens=None, doc_ids=None, doc_ids_k=None, q_offset=0, return_lse=False, out=None, lse=None,
                workspace=None, stream=None):
    """Attention forward with modified scores; q, k, v, tensor_layout, sm_scale, out and lse as ``sage_attn``.

        s = sm_scale q·k;  softcap > 0: s = softcap·tanh(s / softcap);  slopes: s -= slopes[h]·|i + q_offset - j|

    Key j is visible to query i when (not is_causal, or j <= i + q_offset, or j < prefix_lens[b]) and, with
    documents, doc_ids[b, i] == doc_ids_k[b, j] >= 0. ``slopes`` fp32 [Hq]; ``prefix_lens`` int32 [B], with
    is_causal; ``doc_ids`` int32 [B, Nq] and ``doc_ids_k`` int32 [B, Nk] (default: doc_ids, Nq == Nk). A negative
    id is padding. Rows of k and v that are padding, or that lie behind the last key any row sees under the causal
    and prefix masks, may hold anything; all others must be finite in v. ``q_offset``: how many keys lie before the first
    query (the next chunk of a prompt); positions and, with slopes, distances beyond 2^31 - 256 are refused. A row that
    sees no key gives 0 and lse -inf.
    Returns out, plus lse [B, Hq, Nq] fp32 if return_lse."""
    _check_dense_args(q, k, v, tensor_layout, out, lse, return_lse, workspace)
    B, hq, hkv, nq, nk, d = _dims(q, k, tensor_layout)
    index = q.get_device()
    if doc_ids is None and doc_ids_k is not None:
        raise ValueError("doc_ids_k needs doc_ids")
    if doc_ids is not None:
        if doc_ids_k is None:
            if nq != nk:
                raise ValueError("with Nq != Nk the keys' documents need doc_ids_k")
            doc_ids_k = doc_ids
        _check_small("doc_ids", doc_ids, (B, nq), torch.int32, index)
        _check_small("doc_ids_k", doc_ids_k, (B, nk), torch.int32, index)
    if prefix_lens is not None:
        if not is_causal:
            raise ValueError("prefix_lens needs is_causal")
        _check_small("prefix_lens", prefix_lens, (B,), torch.int32, index)
    if slopes is not None:
        _check_small("slopes", slopes, (hq,), torch.float32, index)
    if not -2 ** 31 < q_offset < 2 ** 31:
        raise ValueError("q_offset must fit in 32 bits")
    if not return_lse:
        lse = None
    lib = _lib.load()
    with _Launch(index, stream) as on:
        if out is None:
            out = torch.empty_like(q)
        if return_lse and lse is None:
            lse = torch.empty((B, hq, nq), dtype=torch.float32, device=q.device)
        (qv, q_ok), (kv, k_ok), (vv, v_ok), (ov, _) = (_view(t, d % 8 == 0) for t in (q, k, v, out))
        nbytes = 0 if workspace is not None else scored_attn_workspace_bytes(B, hq, hkv, nq, nk, d, q_ok and k_ok and v_ok,
                                                                             doc_ids is not None)
        with _Scratch(workspace, nbytes, on) as w:
            st = lib.sage_scored_attn(byref(qv), byref(kv), byref(vv), byref(ov), _ptr(lse),
                                      _ptr(slopes), _ptr(prefix_lens), _ptr(doc_ids), _ptr(doc_ids_k), B, hq, hkv, nq, nk, d,
                                      DTYPE[q.dtype], LAYOUT[tensor_layout], bool(is_causal),
                                      _NAN if sm_scale is None else sm_scale, softcap, q_offset, bool(return_lse),
                                      w.at, w.nbytes, on)
    if st:
        raise SageError(st, "scored_attn")
    return (out, lse) if return_lse else out
