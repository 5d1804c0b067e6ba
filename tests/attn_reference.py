"""Attention with modified scores in float64, and how far a kernel may be from it.

The bounds count roundings. A score is a sum of d products in fp32 (each addition off by at most one
step, 2^-23 of the sum of magnitudes), scaled, capped and biased in fp32; `ds` bounds its error. A
softmax weight is then off by a factor of at most e^(2 ds) (its score and its row's sum) and by the
exponential's 2^-22, and is rounded once to the operands' type (half a step, eps / 2). The sum over
the keys is fp32 and the result is rounded once."""

import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, sm_scale, cap=0.0, bias=None, seen=None, dtype=torch.bfloat16, relative_cap=False):
    """q [..., M, d], k / v [..., N, d] (any 16-bit or float type), bias / seen [..., M, N].
    Returns dict(out, lse, p, out_tol, lse_tol, p_tol) in float64."""
    q, k, v = q.double(), k.double(), v.double()
    s = q @ k.transpose(-1, -2) * sm_scale
    size = (q.abs() @ k.abs().transpose(-1, -2)) * sm_scale
    ds = size * (q.shape[-1] + 4) * 2.0 ** -23
    if cap:
        s = cap * torch.tanh(s / cap)
        # tanh to two steps of its range, the scaling around it; relative_cap: scores far below the cap, which
        # are held to eight steps of themselves
        ds = ds + (s.abs() * 2.0 ** -20 if relative_cap else cap * 2.0 ** -21)
    if bias is not None:
        ds = ds + (bias.abs() + s.abs()) * 2.0 ** -22
        s = s + bias
    if seen is None:
        seen = torch.ones_like(s, dtype=torch.bool)
    s = torch.where(seen, s, -math.inf)
    ds = torch.where(seen, ds, 0.0).amax(-1)
    # the base-2 score, its maximum and their difference are fp32 values: a step of the largest of them
    top = torch.where(seen, s.abs(), 0.0).amax(-1)
    ds = ds + top * 1.5 * 2.0 ** -22 + 2.0 ** -22
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    v = torch.where(torch.isfinite(v), v, 0.0)
    out, mag = p @ v, p @ v.abs()
    half = HALF_STEP[dtype]
    w = torch.expm1(2 * ds)[..., None] + 2.0 ** -21 + half
    # fp16's smallest weights round to multiples of 2^-24 rather than relative to themselves
    tiny = 2.0 ** -24 * v.abs().sum(-2, keepdim=True) if dtype == torch.float16 else 0.0
    out_tol = mag * w + half * (out.abs() + mag * w) + tiny + 1e-7
    return dict(out=out, lse=lse, p=p, out_tol=out_tol, lse_tol=ds + (lse.abs() * 2.0 ** -23).nan_to_num(posinf=0.0) + 2.0 ** -21,
                p_tol=p * (torch.expm1(2 * ds)[..., None] + 2.0 ** -21))


def assert_close(got, want, tol, what):
    got = got.double().cpu()
    want, tol = want.cpu(), tol.cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite in other places"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{what}: infinities differ"
    over = (got - want).abs()[fin] / tol[fin]
    assert over.numel() == 0 or over.max() <= 1, f"{what}: {over.max():.3g} of the tolerance"
