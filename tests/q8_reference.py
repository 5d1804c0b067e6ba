"""An 8-bit paged cache on the CPU: its scales and codes by plain loops, and attention over its values in float64
with a bound of how far a kernel may be from it."""

import math

import torch

import paged_reference as ref

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = 2.0 ** -100


def needed(most, dtype):
    """Scale that a largest magnitude (a float32 scalar tensor) needs."""
    if dtype == torch.int8:
        s = most / torch.tensor(127.0)
    else:
        s = torch.tensor(0.0)
        if most > 0:
            e = math.floor(math.log2(float(most))) - 10
            while float(most) > 448.0 * 2.0 ** e:
                e += 1
            s = torch.tensor(2.0 ** e)
    return torch.maximum(s.float(), torch.tensor(LEAST))


def to_codes(u, dtype):
    return u.round().clamp(-127, 127).to(torch.int8) if dtype == torch.int8 else u.to(dtype)


def make_cache(lens, hkv, d, page, block, kt, vt, layout="HND", seed=0, room=0, spread=0.0):
    """A cache of random codes and scales (positive; `spread`: of their base-2 logarithm)."""
    c = ref.make_cache(lens, hkv, d, page, torch.float32, layout, seed=seed, room=room)
    g = torch.Generator().manual_seed(seed + 77)
    shape = (c["k"].shape[0], hkv, page // block)
    for w, t in (("k", kt), ("v", vt)):
        x = c[w] * (40.0 if t == torch.int8 else 60.0)
        c[w] = to_codes(x, t)
        c[w + "s"] = torch.exp2(torch.randn(shape, generator=g) * spread) * 0.02
    c["block"] = block
    return c


def get(c, which, page, h, slot):
    """Codes of one row, in their type."""
    x = c[which].view(torch.uint8)
    row = x[page, h, slot] if c["layout"] == "HND" else x[page, slot, h]
    return row.view(c[which].dtype)


def put(c, which, page, h, slot, codes):
    ref.set_row({which: c[which].view(torch.uint8), "layout": c["layout"]}, which, page, h, slot, codes.view(torch.uint8))


def values(c, which, b, h, n, first=0):
    """Values of slots first .. n - 1 of sequence b, [tokens, d] float64; exact."""
    t = torch.arange(first, n)
    p, s = c["table"][b, t // c["size"]].long(), t % c["size"]
    x = c[which].view(torch.uint8)
    x = (x[p, h, s] if c["layout"] == "HND" else x[p, s, h]).view(c[which].dtype)
    return x.float().double() * c[which + "s"][p, h, s // c["block"]].double()[:, None]


def append(c, k, v, cu=None):
    """In place: tokens that have a place (the caller gives no others)."""
    batch, hkv = c["table"].shape[0], k.shape[1]
    cu = list(range(batch + 1)) if cu is None else cu
    for which, x in (("k", k), ("v", v)):
        dt = c[which].dtype
        for b in range(batch):
            held, new = int(c["lens"][b]), cu[b + 1] - cu[b]
            t = held
            while t < held + new:
                end = min(held + new, (t // c["block"] + 1) * c["block"])
                page, s0 = int(c["table"][b, t // c["size"]]), t % c["size"]
                block, inside = s0 // c["block"], s0 % c["block"]
                for h in range(hkv):
                    rows = x[cu[b] + t - held:cu[b] + end - held, h].float()
                    was = c[which + "s"][page, h, block].clone() if inside else torch.tensor(0.0)
                    scale = torch.maximum(was, needed(rows.abs().max(), dt))
                    if inside and scale > was:
                        f = was / scale
                        for i in range(inside):
                            old = get(c, which, page, h, s0 - inside + i).float()
                            put(c, which, page, h, s0 - inside + i, to_codes(old * f, dt))
                    inv = torch.tensor(1.0) / scale
                    for i in range(end - t):
                        put(c, which, page, h, s0 + i, to_codes(rows[i] * inv, dt))
                    c[which + "s"][page, h, block] = scale
                t = end


def attend(c, q, sm_scale, cap=0.0, slopes=None, qpos=None, hkv=1):
    """dict(out, lse, out_tol, lse_tol) of one query per sequence, in float64.

    The bound: a score is a sum of d products in fp32 (each addition off by at most a step of 2^-23 of the sum of
    magnitudes; q as fp16 of a scaled row is exact but for channels below 2^-38 of its largest), times two factors, capped,
    biased. A weight is off by e^(2 ds) by its score and its sum, by the exponentials and the logarithm of the scale
    (2^-20 together) and by its rounding to fp16, half a step of 2^-10; weights below fp16's normal range by half of 2^-24
    in a frame whose largest is at least 2^7. The sum is fp32, the result is rounded once."""
    B, hq, d = q.shape
    g = hq // hkv
    res = dict(out=torch.zeros(B, hq, d, dtype=torch.float64), lse=torch.full((B, hq), -math.inf, dtype=torch.float64),
               out_tol=torch.full((B, hq, d), 1e-12, dtype=torch.float64), lse_tol=torch.ones(B, hq, dtype=torch.float64))
    for b, n in enumerate(c["lens"].tolist()):
        if n == 0:
            continue
        for h in range(hkv):
            at = slice(h * g, (h + 1) * g)
            x, k, v = q[b, at].double(), values(c, "k", b, h, n), values(c, "v", b, h, n)
            s = x @ k.T * sm_scale
            size = x.abs() @ k.abs().T * sm_scale
            ds = size * (d + 8) * 2.0 ** -23 + x.abs().amax(-1, keepdim=True) * k.abs().sum(-1) * sm_scale * 2.0 ** -38
            if cap:
                s = cap * torch.tanh(s / cap)
                ds = ds + cap * 2.0 ** -21
            if slopes is not None:
                here = n - 1 if qpos is None else int(qpos[b])
                bias = -slopes[at, None].double() * (here - torch.arange(n).double()).abs()
                ds = ds + (bias.abs() + s.abs()) * 2.0 ** -22
                s = s + bias
            ds = ds.amax(-1) + s.abs().amax(-1) * 1.5 * 2.0 ** -22 + 2.0 ** -22
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, None])
            out, mag = p @ v, p @ v.abs()
            w = torch.expm1(2 * ds)[:, None] + 2.0 ** -20 + 2.0 ** -11
            scale = values(dict(c, v=torch.ones_like(c["v"].float()).to(c["v"].dtype)), "v", b, h, n)[:, 0]
            tiny = 2.0 ** -32 * (p * scale).amax(-1, keepdim=True) * (v.abs() / scale[:, None].clamp(min=1e-300)).sum(0)
            half = HALF_STEP[q.dtype]
            res["out"][b, at], res["lse"][b, at] = out, lse
            err = mag * w + tiny
            least = 2.0 ** -25 if q.dtype == torch.float16 else 0.0  # half of the smallest fp16
            res["out_tol"][b, at] = err + half * (out.abs() + err) + least + 1e-12
            res["lse_tol"][b, at] = ds + lse.abs() * 2.0 ** -23 + 2.0 ** -20
    return res
