"""Norms and rotation of queries and keys against float64, with angles from exact fractions."""

import math
from fractions import Fraction

import pytest
import torch

from attn_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# 2 pi to 60 digits
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def angles(positions, freq):
    """cos and sin of position * freq, the angle reduced in exact arithmetic."""
    f = [Fraction(float(x)) / TWO_PI for x in freq]
    rows = []
    for p in positions.flatten().tolist():
        rows.append([float((p * x) % 1) * 2 * math.pi for x in f])
    a = torch.tensor(rows, dtype=torch.float64).view(*positions.shape, len(f))
    return torch.cos(a), torch.sin(a)


def reference(x, w, positions, freq, eps, interleaved):
    """x [..., tokens, heads, d], positions [..., tokens]; (value, bound)."""
    y = x.double()
    y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    d, n = x.shape[-1], 0 if freq is None else freq.numel()
    out, mag = y.clone(), y.abs()
    if n:
        cos, sin = (t[..., None, :] for t in angles(positions, freq))
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        a, b = y[..., i], y[..., j]
        out[..., i], out[..., j] = a * cos - b * sin, b * cos + a * sin
        both = a.abs() + b.abs()
        mag[..., i], mag[..., j] = both, both
    # the sum of squares is off by a step per addition, half of which the root leaves; its reciprocal, the factors and
    # the rotation by a step or two each; cos and sin by 2^-21 (their own step and that of the angle, at most pi, in fp32)
    err = mag * ((d / 2 + 12) * 2.0 ** -23 + 2.0 ** -21)
    half = HALF_STEP[x.dtype]
    least = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    return out, err + half * (out.abs() + err) + least + 1e-30


def freqs(n, base=10000.0):
    return (base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))).float()


CASES = [
    # tokens, hq, hkv, d, pairs of channels, dtype, interleaved, weight type
    (1, 1, 1, 64, 32, torch.float16, False, None),
    (7, 32, 8, 128, 64, torch.bfloat16, False, torch.bfloat16),
    (130, 5, 3, 128, 32, torch.bfloat16, False, torch.float32),       # half of the channels
    (33, 4, 2, 72, 18, torch.float16, True, torch.float16),
    (9, 3, 1, 72, 36, torch.float16, False, torch.float16),           # runs of 4
    (9, 3, 1, 36, 18, torch.bfloat16, False, torch.float32),          # runs of 2
    (11, 2, 2, 33, 16, torch.float16, False, torch.float16),          # channel by channel, an odd one over
    (11, 2, 2, 127, 63, torch.bfloat16, True, torch.float32),
    (5, 3, 1, 127, 63, torch.float16, False, None),
    (5, 3, 1, 120, 7, torch.bfloat16, True, None),                    # pairs end inside a run
    (5, 3, 1, 80, 40, torch.bfloat16, False, torch.bfloat16),
    (5, 3, 1, 1, 0, torch.float16, False, torch.float16),
    (3, 2, 1, 2, 1, torch.float16, False, torch.float32),
    (40, 2, 2, 96, 0, torch.bfloat16, False, torch.bfloat16),         # norms alone
    (5000, 2, 1, 64, 32, torch.float16, True, torch.float16),
]


@pytest.mark.parametrize("tokens,hq,hkv,d,pairs,dtype,interleaved,wtype", CASES)
def test_packed(tokens, hq, hkv, d, pairs, dtype, interleaved, wtype):
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(tokens + d)
    q, k = (torch.randn(tokens, h, d, generator=g).mul(torch.rand(tokens, h, 1, generator=g) * 8).to(dtype) for h in (hq, hkv))
    w = [None, None] if wtype is None else [(1 + 0.3 * torch.randn(d, generator=g)).to(wtype) for _ in "qk"]
    pos = torch.randint(0, 5000, (tokens,), generator=g, dtype=torch.int32)
    freq = freqs(pairs) if pairs else None
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got = qa.qk_norm_rope(on(q), on(k), on(pos), on(freq), on(w[0]), on(w[1]), eps=1e-5, interleaved=interleaved)
    for name, x, y, wx in zip("qk", (q, k), got, w):
        want, tol = reference(x, wx, pos, freq, 1e-5, interleaved)
        assert y.dtype == dtype and y.is_contiguous()
        assert_close(y, want, tol, name)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("per_row", [False, True])
def test_slices_of_one_projection_in_place(layout, per_row):
    import quantized_attention_mean_gb300 as qa
    B, N, hq, hkv, d = 2, 37, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(B, N, hq + 2 * hkv, d, generator=g).bfloat16()
    pos = torch.randint(-50, 9000, (B, N) if per_row else (N,), generator=g, dtype=torch.int32)
    freq = freqs(32)
    x = rows.to(DEV)
    q, k = x[:, :, :hq], x[:, :, hq:hq + hkv]
    if layout == "HND":
        q, k = q.transpose(1, 2), k.transpose(1, 2)
    fresh = qa.qk_norm_rope(q, k, pos.to(DEV), freq.to(DEV), tensor_layout=layout)
    wide = torch.full((B, N, hq + hkv, d), 5.0, dtype=torch.bfloat16, device=DEV)
    apart = [wide[:, :, :hq], wide[:, :, hq:]]
    if layout == "HND":
        apart = [t.transpose(1, 2) for t in apart]
    qa.qk_norm_rope(q, k, pos.to(DEV), freq.to(DEV), tensor_layout=layout, q_out=apart[0], k_out=apart[1])
    a, b = qa.qk_norm_rope(q, k, pos.to(DEV), freq.to(DEV), tensor_layout=layout, q_out=q, k_out=k)
    assert a is q and b is k
    assert torch.equal(x[:, :, hq + hkv:].cpu(), rows[:, :, hq + hkv:])          # the values beside them stay
    at = pos if per_row else pos.expand(B, N)
    for name, part, outs in (("q", rows[:, :, :hq], (fresh[0], apart[0], q)), ("k", rows[:, :, hq:hq + hkv], (fresh[1], apart[1], k))):
        want, tol = reference(part, None, at, freq, 1e-6, False)
        for y in outs:
            assert_close(y.transpose(1, 2) if layout == "HND" else y, want, tol, name)


def test_odd_addresses_and_broadcast_inputs():
    # rows that begin at any element, a key that all heads share, positions that count by themselves
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(8)
    wide = torch.randn(20, 3, 65, generator=g).half()
    one = torch.randn(20, 1, 64, generator=g).half()
    freq = freqs(32)
    w = wide.to(DEV)
    q, k = qa.qk_norm_rope(w[..., 1:], one.to(DEV).expand(20, 4, 64), None, freq.to(DEV))
    at = torch.arange(20)
    for name, y, x in (("q", q, wide[..., 1:]), ("k", k, one.expand(20, 4, 64))):
        want, tol = reference(x, None, at, freq, 1e-6, False)
        assert_close(y, want, tol, name)


@pytest.mark.parametrize("base", [10000.0, 5e6])
def test_far_positions(base):
    import quantized_attention_mean_gb300 as qa
    pos = torch.tensor([0, 1, -1, 4097, 2 ** 20 + 3, 2 ** 24 + 1, -2 ** 30 - 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(9, 2, 128, generator=g).half()
    freq = freqs(64, base)
    for f in (freq, -freq, freq * 3.0):
        out, _ = qa.qk_norm_rope(q.to(DEV), q.to(DEV), pos.to(DEV), f.to(DEV))
        want, tol = reference(q, None, pos, f, 1e-6, False)
        # inv_freq / 2 pi in 64 bits, off by a step of itself, times the position
        turn = 2.0 ** -52 * f.double().abs().max() * pos.double().abs()[:, None, None]
        assert_close(out, want, tol + turn * q.double().abs().amax() * 4, "q")


def test_zero_rows_and_large_values():
    import quantized_attention_mean_gb300 as qa
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q[1] = 1e15
    q[2, :, 0] = 3e-20
    freq = freqs(32)
    out, _ = qa.qk_norm_rope(q.to(DEV), q.to(DEV), None, freq.to(DEV), eps=1e-6)
    want, tol = reference(q, None, torch.arange(3), freq, 1e-6, False)
    assert_close(out, want, tol, "q")
    assert (out[0] == 0).all()


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -100, 1e-6])
@pytest.mark.parametrize("hq,hkv,d,pairs,interleaved", [(5, 3, 64, 32, False), (3, 1, 128, 64, True), (16, 2, 36, 9, False), (2, 2, 33, 16, True)])
def test_rows_of_every_magnitude(hq, hkv, d, pairs, interleaved, eps):
    # rows from the smallest bf16 on, beside ordinary ones: where eps does not outweigh them, squares that leave fp32 on either side
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(d)
    sizes = [1.0, 1e-10, 1e-18, 1e-21, 1e-25, 1e-38, 2e-40, 1e10, 1e17, 1e19, 1e25, 3e37]
    if eps > 2.0 ** -90:
        sizes = sizes[:9]                                               # (magnitudes below 1e18)
    T = 4 * len(sizes)
    q, k = (torch.randn(T, h, d, generator=g).clamp(-8, 8) for h in (hq, hkv))
    order = torch.randperm(T * hq, generator=g)[:T * hq].view(T, hq) % len(sizes)
    q = (q.double() * torch.tensor(sizes, dtype=torch.float64)[order][..., None]).bfloat16()
    k = (k.double() * torch.tensor(sizes, dtype=torch.float64)[torch.arange(T) % len(sizes)][:, None, None]).bfloat16()
    q[3, 0, 1:] = 0                                                     # one value of its row, as large as it gets
    q[3, 0, 0] = torch.finfo(torch.bfloat16).max if eps < 2.0 ** -90 else 1e17
    for x in (q, k):                                                    # (a row of zeros has no value with eps = 0)
        x[..., 0] = torch.where((x == 0).all(-1), torch.tensor(2.0 ** -133).bfloat16(), x[..., 0])
    w = (1 + 0.3 * torch.randn(d, generator=g)).float()
    pos, freq = torch.arange(T, dtype=torch.int32), freqs(pairs)
    a, b = q.to(DEV), k.to(DEV)
    got = qa.qk_norm_rope(a, b, pos.to(DEV), freq.to(DEV), w.to(DEV), w.to(DEV), eps=eps, interleaved=interleaved)
    for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
        want, tol = reference(x, w, pos, freq, eps, interleaved)
        assert_close(y, want, tol + 2.0 ** -126, name)                  # (results below bf16's normal range may become 0)
    qa.qk_norm_rope(a, b, pos.to(DEV), freq.to(DEV), w.to(DEV), w.to(DEV), eps=eps, interleaved=interleaved, q_out=a, k_out=b)
    assert torch.equal(a, got[0]) and torch.equal(b, got[1])


def test_empty_and_on_another_stream_and_captured():
    import quantized_attention_mean_gb300 as qa
    freq = freqs(32).to(DEV)
    e = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    a, b = qa.qk_norm_rope(e, e, None, freq)
    assert a.shape == b.shape == (0, 4, 64)
    q = torch.randn(300, 8, 64, dtype=torch.float16, device=DEV)
    k = torch.randn(300, 2, 64, dtype=torch.float16, device=DEV)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    want = qa.qk_norm_rope(q, k, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qa.qk_norm_rope(q, k, pos, freq, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = qa.qk_norm_rope(q, k, pos, freq)
    q2 = torch.randn_like(q)
    q.copy_(q2)
    pos.add_(1000)
    graph.replay()
    want = qa.qk_norm_rope(q2, k, pos, freq)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, want))
