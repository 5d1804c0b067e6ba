"""Norms of queries and keys for each head and their rotation by position, in one pass: what stands between a
layer's projections and its attention call or cache."""

from ctypes import byref

import torch

from . import DTYPE, LAYOUT, SageError, _lib
from ._lib import SageView
from .paged import _check_range, _check_small, _Launch, _ptr

__all__ = ["qk_norm_rope"]

F32 = 2  # SAGE_F32


def _check_weight(name, w, d, dtype, index):
    if (w.dtype != dtype and w.dtype != torch.float32) or w.shape != (d,) or w.get_device() != index or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{d}] tensor of q's dtype or float32 on q's device")


def _view(t, packed, hnd):
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    if packed:
        return SageView(t.data_ptr(), 0, st[0], st[1])
    return SageView(t.data_ptr(), st[0], st[1], st[2])


def _apart(x, y):
    """Whether no element of x is one of y: apart as a whole, or interleaved, as slices of one projection's rows are."""
    if x.numel() == 0 or y.numel() == 0:
        return True
    dims = [[(n, s) for n, s in zip(t.shape, t.stride()) if n > 1] for t in (x, y)]
    size, gap = x.element_size(), y.data_ptr() - x.data_ptr()
    spans = [1 + sum((n - 1) * s for n, s in d) for d in dims]
    if gap >= spans[0] * size or -gap >= spans[1] * size:
        return True
    # modulo some pitch, of which all longer strides are multiples, both are runs that do not meet
    for pitch in {s for d in dims for _, s in d if s > 1}:
        if gap % size or any(s >= pitch and s % pitch for d in dims for _, s in d):
            continue
        runs = [1 + sum((n - 1) * s for n, s in d if s < pitch) for d in dims]
        at = gap // size % pitch
        if runs[0] <= at and at + runs[1] <= pitch:
            return True
    return False


def _same(x, y):
    return x.data_ptr() == y.data_ptr() and x.shape == y.shape and x.stride() == y.stride()


def _check_outputs(q, k, q_out, k_out, dtype, index):
    for name, out, t in (("q_out", q_out, q), ("k_out", k_out, k)):
        if out is not None:
            if out.shape != t.shape or out.dtype != dtype or out.get_device() != index:
                raise ValueError(f"{name} must have its input's shape, dtype and device")
            # rows are read once each, at any time: an output is its own input or lies apart from both
            for x in (q, k):
                if not (x is t and _same(out, t)) and not _apart(out, x):
                    raise ValueError(f"{name} must be its input itself or not overlap an input")
    if q_out is not None and k_out is not None and not _apart(q_out, k_out):
        raise ValueError("q_out and k_out must not overlap")


def qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, tensor_layout="NHD",
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """For each (token, head) row of q and k: ``y = x / sqrt(mean(x²) + eps) · weight``, then the first
    ``2 · len(inv_freq)`` channels rotated by ``position · inv_freq[p]``: the pairs (p, p + len(inv_freq)), or
    (2p, 2p + 1) if ``interleaved``, become ``(a cos − b sin, b cos + a sin)``. Returns (q_out, k_out), new tensors
    unless given; an output may be its input (in place).

    q: [tokens, Hq, d] packed, or [B, N, Hq, d] / [B, Hq, N, d] by ``tensor_layout`` ("NHD" / "HND"); k: Hkv heads of
    the same tokens; fp16 or bf16, head_dim up to 128, any strides but the last (slices of one projection's output).
    ``positions``: int32 [tokens], or [N] or [B, N]; default: the token's index. ``inv_freq``: float32, at most d / 2;
    without it nothing is rotated. Weights: [d], q's dtype or float32; default: ones. Arithmetic is in fp32 (magnitudes
    below 1e18, with eps below 2^-90 any; down to the smallest), rounded once at the end; angles are
    taken in 64 bits, off by at most 2^-52 of themselves and 2^-65 of a turn per position (5e-7 · inv_freq + 4e-10 at 2^31)."""
    if tensor_layout not in LAYOUT:
        raise ValueError("tensor_layout must be 'HND' or 'NHD'")
    shape, other = q.shape, k.shape
    dims, dtype = len(shape), q.dtype
    if (dims != 3 and dims != 4) or len(other) != dims:
        raise ValueError("q and k must be packed [tokens, heads, head_dim] or 4-D tensors")
    if dtype not in DTYPE or k.dtype != dtype:
        raise TypeError("q and k must share one dtype, float16 or bfloat16")
    packed, hnd = dims == 3, tensor_layout == "HND"
    if packed:
        if hnd:
            raise ValueError("packed rows are [tokens, heads, head_dim]: tensor_layout 'NHD'")
        B, Bk, (N, hq, d), (Nk, hkv, dk) = 1, 1, shape, other
    elif hnd:
        (B, hq, N, d), (Bk, hkv, Nk, dk) = shape, other
    else:
        (B, N, hq, d), (Bk, Nk, hkv, dk) = shape, other
    if Bk != B or Nk != N or dk != d:
        raise ValueError("k must have q's tokens and head_dim")
    index = q.get_device()
    if k.get_device() != index:
        raise ValueError("q and k must be on one CUDA device")
    wtype = dtype
    if q_weight is not None:
        _check_weight("q_weight", q_weight, d, dtype, index)
        wtype = q_weight.dtype
    if k_weight is not None:
        _check_weight("k_weight", k_weight, d, dtype, index)
        if q_weight is not None and k_weight.dtype != wtype:
            raise TypeError("q_weight and k_weight must share one dtype")
        wtype = k_weight.dtype
    rot = 0
    if inv_freq is not None:
        _check_small("inv_freq", inv_freq, (inv_freq.numel(),), torch.float32, index)
        rot = 2 * inv_freq.numel()
        if rot > d:
            raise ValueError("inv_freq must have at most head_dim / 2 entries")
    by_row = 0
    if positions is not None:
        by_row = N if positions.dim() == 2 else 0
        _check_small("positions", positions, (B, N) if positions.dim() == 2 and not packed else (N,), torch.int32, index)
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps must be finite and not negative")
    if q_out is not None or k_out is not None:
        _check_outputs(q, k, q_out, k_out, dtype, index)
    if index < 0:
        raise ValueError("q and k must be on a CUDA device")
    _check_range("the number of tokens", B * N)
    with _Launch(index, stream) as on:
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=q.device)
        if k_out is None:
            k_out = torch.empty(other, dtype=dtype, device=q.device)
        code = DTYPE[dtype]
        st = _lib.load().sage_qk_norm_rope(byref(_view(q, packed, hnd)), byref(_view(k, packed, hnd)),
                                           byref(_view(q_out, packed, hnd)), byref(_view(k_out, packed, hnd)), _ptr(positions),
                                           by_row, _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight),
                                           code if wtype == dtype else F32, B, hq, hkv, N, d, rot, code, LAYOUT[tensor_layout],
                                           bool(interleaved), eps, on)
    if st:
        raise SageError(st, "qk_norm_rope")
    return q_out, k_out
