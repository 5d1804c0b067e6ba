"""Attention with modified scores against float64: caps, distance bias, causal, prefix and document
masks, at the sizes where tiles, splits and layouts end."""

import math

import pytest
import torch

from attn_reference import assert_close, attend

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def docs_of(lengths, pad, B=1, shuffle=False, seed=0):
    ids = torch.cat([torch.full((n,), i) for i, n in enumerate(lengths)] + [torch.full((pad,), -1)]).to(torch.int32)
    ids = ids[None].repeat(B, 1)
    if shuffle:
        g = torch.Generator().manual_seed(seed)
        ids = torch.stack([r[torch.randperm(r.numel(), generator=g)] for r in ids])
    return ids.contiguous()


def visible(nq, nk, B, causal, offset, prefix, dq, dk):
    i, j = torch.arange(nq)[:, None] + offset, torch.arange(nk)[None]
    seen = torch.ones(B, nq, nk, dtype=torch.bool)
    if causal:
        seen = (j <= i)[None].expand(B, nq, nk).clone()
        if prefix is not None:
            seen |= (j[None] < prefix[:, None, None])
    if dq is not None:
        seen &= (dq[:, :, None] == dk[:, None, :]) & (dk[:, None, :] >= 0)
    return seen


def check(B, hq, hkv, nq, nk, d, dtype, layout="HND", causal=False, cap=0.0, bias=False, prefix=None, dq=None, dk=None,
          offset=0, scale=None, q=None, k=None, v=None, place=None, clean=None, seed=0, relative_cap=False):
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(seed + nq + d)
    q = (torch.randn(B, hq, nq, d, generator=g) * 2).to(dtype) if q is None else q
    k = torch.randn(B, hkv, nk, d, generator=g).to(dtype) if k is None else k
    v = torch.randn(B, hkv, nk, d, generator=g).to(dtype) if v is None else v
    slopes = 2.0 ** (-torch.arange(1, hq + 1).float() * 8 / hq) if bias else None
    prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    dk = dq if dk is None else dk
    gpu = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    lay = lambda t: gpu(t if layout == "HND" else t.transpose(1, 2).contiguous())  # noqa: E731
    lay = place or lay
    ws = qa.alloc_workspace(qa.scored_attn_workspace_bytes(B, hq, hkv, nq, nk, d, packed=False), DEV)
    ws.fill_(255)
    out, lse = qa.scored_attn(lay(q), lay(k), lay(v), tensor_layout=layout, is_causal=causal, softcap=cap, sm_scale=scale,
                              slopes=gpu(slopes), prefix_lens=gpu(prefix), doc_ids=gpu(dq), doc_ids_k=gpu(dk),
                              q_offset=offset, return_lse=True, workspace=ws)
    assert qa.read_device_status(ws) == 0
    seen = visible(nq, nk, B, causal, offset, prefix, dq, dk)[:, None]
    grp = hq // hkv
    kk, vv = (t.repeat_interleave(grp, 1).to(DEV) for t in (k, v if clean is None else clean))
    if clean is not None:
        kk = torch.where(torch.isfinite(kk.float()), kk, torch.zeros_like(kk))
    b = None
    if bias:
        dist = (torch.arange(nq)[:, None] + offset - torch.arange(nk)).abs().double()
        b = (-slopes.double()[:, None, None] * dist)[None].to(DEV)
    r = attend(q.to(DEV), kk, vv, d ** -0.5 if scale is None else scale, cap, b, seen.expand(B, hq, nq, nk).to(DEV), dtype, relative_cap)
    o = out if layout == "HND" else out.transpose(1, 2)
    assert_close(o, r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")
    return out, lse


F, H = torch.float16, torch.bfloat16
SIZES = [
    # B, hq, hkv, nq, nk, d, dtype, layout
    (1, 1, 1, 1, 1, 64, F, "HND"),
    (2, 4, 2, 1, 130, 128, H, "NHD"),
    (1, 2, 1, 128, 128, 64, H, "HND"),
    (1, 2, 2, 129, 127, 128, F, "HND"),
    (2, 3, 1, 257, 400, 64, F, "NHD"),
    (1, 2, 2, 300, 513, 72, H, "HND"),
    (1, 4, 4, 65, 1000, 96, F, "NHD"),
    (1, 2, 1, 50, 70, 33, F, "HND"),       # rows that TMA cannot address
    (2, 2, 1, 140, 140, 20, H, "NHD"),
    (1, 2, 2, 700, 700, 8, H, "HND"),
]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (15.0, False), (0.0, True), (15.0, True)])
def test_full(size, cap, bias):
    B, hq, hkv, nq, nk, d, dtype, layout = size
    check(B, hq, hkv, nq, nk, d, dtype, layout, cap=cap, bias=bias)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_causal_with_offset(size, cap, bias):
    B, hq, hkv, nq, nk, d, dtype, layout = size
    for offset in {0, nk - nq, -5, nk}:
        check(B, hq, hkv, nq, nk, d, dtype, layout, causal=True, cap=cap, bias=bias, offset=offset)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (10.0, False), (0.0, True), (10.0, True)])
@pytest.mark.parametrize("d,dtype", [(64, H), (128, F)])
def test_prefix(cap, bias, d, dtype):
    for prefix in ([0, 300, 77], [128, 1, 299], [-4, 1000, 129]):
        check(3, 2, 1, 300, 300, d, dtype, causal=True, prefix=prefix, cap=cap, bias=bias)
    check(1, 2, 1, 100, 900, d, dtype, causal=True, prefix=[640], offset=3, cap=cap, bias=bias)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("d,dtype,layout", [(64, F, "NHD"), (128, H, "HND")])
@pytest.mark.parametrize("causal", [False, True])
def test_documents(cap, bias, d, dtype, layout, causal):
    for lengths, pad in (([600], 0), ([1, 127, 128, 129, 200], 15), ([300, 5, 5, 5, 200], 130), ([], 600), ([7] * 80, 40)):
        dq = docs_of(lengths, pad, 2)
        check(2, 2, 1, dq.shape[1], dq.shape[1], d, dtype, layout, causal=causal, cap=cap, bias=bias, dq=dq)
    dq = docs_of([200, 100, 30], 20, 2, shuffle=True)
    check(2, 2, 1, 350, 350, d, dtype, layout, causal=causal, cap=cap, bias=bias, dq=dq)
    # other documents on the key side, some of them nobody's
    dk = docs_of([50, 0, 120, 300], 33, 1)
    check(1, 2, 1, 300, dk.shape[1], d, dtype, layout, cap=cap, bias=bias, dq=docs_of([100, 100, 90], 10, 1), dk=dk)
    # with a prefix
    check(2, 2, 1, 350, 350, d, dtype, layout, causal=True, cap=cap, bias=bias, dq=docs_of([200, 150], 0, 2),
          prefix=[140, 260])


@pytest.mark.parametrize("nq,nk,hq", [(1, 20000, 2), (100, 9001, 4), (128, 4096, 1), (300, 2500, 1), (5, 513, 1)])
@pytest.mark.parametrize("d,dtype", [(64, F), (128, H)])
def test_few_rows_are_split_over_the_keys(nq, nk, hq, d, dtype):
    check(1, hq, 1, nq, nk, d, dtype, causal=True, offset=nk - nq)
    check(1, hq, 1, nq, nk, d, dtype, causal=True, offset=nk // 3, bias=True, cap=12.0)
    # one of the keys' documents, from somewhere in their middle, and padding
    check(1, hq, 1, nq, nk, d, dtype, "NHD", dq=torch.full((1, nq), 1, dtype=torch.int32),
          dk=docs_of([nk // 3, nk - nk // 3 - 9], 9, 1))


# CTAs that walk many key tiles without a split: rings of stages and barrier phases that turn many times, the near-to-far
# order, the shorter walk of the first query tile; some rows of each warp against float64
@pytest.mark.parametrize("n,nk,d,dtype,layout,kw", [
    (8192, 8192, 128, H, "HND", dict(causal=True)),
    (8192, 8192, 128, H, "NHD", dict(causal=True, cap=50.0)),
    (8192, 8192, 128, F, "HND", dict(causal=True, bias=True)),
    (8190, 8190, 128, H, "HND", dict(causal=True, cap=12.0, bias=True)),      # scores that reach the cap
    (4000, 9001, 128, F, "NHD", dict(causal=True, offset=5001)),
    (2561, 20001, 128, H, "HND", dict(cap=30.0)),
    (16383, 16383, 128, F, "NHD", dict(causal=True, docs=True)),
    (8192, 8192, 128, H, "HND", dict(causal=True, prefix=4999)),
    (8192, 8192, 64, F, "HND", dict(causal=True)),
    (8192, 8192, 64, H, "NHD", dict(causal=True, cap=50.0)),
    (8191, 8191, 64, H, "HND", dict(causal=True, bias=True)),
    (8192, 8192, 64, F, "HND", dict(causal=True, cap=12.0, bias=True)),
    (16383, 16383, 64, H, "NHD", dict(causal=True, docs=True)),
    (16383, 16383, 64, F, "HND", dict(docs=True, cap=30.0, bias=True)),
    (8192, 8192, 72, H, "NHD", dict(causal=True, prefix=6001, bias=True)),
    (5000, 16001, 40, F, "HND", dict()),
])
def test_long_prompts(n, nk, d, dtype, layout, kw):
    import quantized_attention_mean_gb300 as qa
    hq, hkv = 8, 4
    g = torch.Generator(DEV).manual_seed(n + d)
    q, k, v = (torch.randn(1, h, m, d, generator=g, device=DEV).to(dtype) for h, m in ((hq, n), (hkv, nk), (hkv, nk)))
    q = (q * 2).to(dtype)
    slopes = 2.0 ** (-torch.arange(1, hq + 1, device=DEV).float() * 8 / hq) if kw.get("bias") else None
    prefix = torch.tensor([kw["prefix"]], dtype=torch.int32, device=DEV) if "prefix" in kw else None
    ids = docs_of([1, 5000, 130, 127, 6500, 4000], n - 15758).to(DEV) if kw.get("docs") else None
    causal, offset, cap = kw.get("causal", False), kw.get("offset", 0), kw.get("cap", 0.0)
    lay = lambda t: t if layout == "HND" else t.transpose(1, 2).contiguous()  # noqa: E731
    out, lse = qa.scored_attn(lay(q), lay(k), lay(v), tensor_layout=layout, is_causal=causal, softcap=cap, slopes=slopes,
                              prefix_lens=prefix, doc_ids=ids, q_offset=offset, return_lse=True)
    out = lay(out) if layout == "HND" else out.transpose(1, 2)
    rows = torch.cat([torch.arange(3, n, 61, device=DEV), torch.tensor([0, 127, 128, 255, 256, n - 1], device=DEV)])
    i, j = rows[:, None] + offset, torch.arange(nk, device=DEV)
    seen = (j <= i) if causal else torch.ones(len(rows), nk, dtype=torch.bool, device=DEV)
    if prefix is not None:
        seen = seen | (j < kw["prefix"])
    if ids is not None:
        seen = seen & (ids[0, rows, None] == ids[0]) & (ids[0] >= 0)
    for h in range(hq):
        bias = -slopes[h].double() * (i - j).abs().double() if slopes is not None else None
        r = attend(q[0, h, rows], k[0, h * hkv // hq], v[0, h * hkv // hq], d ** -0.5, cap, bias, seen, dtype)
        assert_close(out[0, h, rows], r["out"], r["out_tol"], f"out of head {h}")
        assert_close(lse[0, h, rows], r["lse"], r["lse_tol"], f"lse of head {h}")


# Few queries of several heads in one query tile or two, groups that do not fill them, splits and none
@pytest.mark.parametrize("B,hq,hkv,nq,nk", [(2, 8, 2, 20, 6000), (2, 14, 2, 16, 6000), (2, 14, 2, 40, 6000),
                                            (1, 32, 8, 100, 9000), (20, 12, 4, 100, 300), (30, 16, 4, 5, 700),
                                            (16, 14, 2, 40, 500), (20, 8, 2, 1, 900), (12, 10, 2, 64, 700),
                                            (1, 40, 2, 3, 2000), (1, 71, 1, 7, 3300), (2, 33, 1, 9, 130)])
@pytest.mark.parametrize("d,dtype,layout", [(64, F, "NHD"), (128, H, "HND"), (40, H, "HND"), (33, F, "NHD")])
def test_heads_share_a_tile(B, hq, hkv, nq, nk, d, dtype, layout):
    g = torch.Generator().manual_seed(nq)
    check(B, hq, hkv, nq, nk, d, dtype, layout, causal=True, offset=nk - nq, bias=True)
    check(B, hq, hkv, nq, nk, d, dtype, layout, causal=True, offset=-3, cap=9.0,
          prefix=torch.randint(0, nk, (B,), generator=g).tolist())
    dk = docs_of([nk // 3, nk - nk // 3 - 9], 9, B)
    check(B, hq, hkv, nq, nk, d, dtype, layout, dq=torch.randint(-1, 3, (B, nq), generator=g, dtype=torch.int32), dk=dk,
          bias=True, cap=20.0)


def test_padding_may_hold_anything():
    dq = docs_of([150, 100], 70, 1)
    g = torch.Generator().manual_seed(3)
    for d, dtype in ((64, F), (128, H)):
        k, v = (torch.randn(1, 2, 320, d, generator=g).to(dtype) for _ in "kv")
        clean = v.clone()
        k[:, :, 250:], v[:, :, 250::2], v[:, :, 251::2] = math.nan, math.inf, math.nan
        clean[:, :, 250:] = 0
        q = torch.randn(1, 2, 320, d, generator=g).to(dtype)
        q[:, :, 250:] = math.nan
        import quantized_attention_mean_gb300 as qa
        for causal in (False, True):
            out, lse = qa.scored_attn(q.to(DEV), k.to(DEV), v.to(DEV), is_causal=causal, doc_ids=dq.to(DEV), return_lse=True)
            kz, qz = torch.nan_to_num(k), torch.nan_to_num(q)
            seen = visible(320, 320, 1, causal, 0, None, dq, dq)[:, None].expand(1, 2, 320, 320).to(DEV)
            r = attend(qz.to(DEV), kz.to(DEV), clean.to(DEV), d ** -0.5, seen=seen, dtype=dtype)
            assert_close(out, r["out"], r["out_tol"], "out")
            assert_close(lse, r["lse"], r["lse_tol"], "lse")
            assert (out[:, :, 250:] == 0).all()


@pytest.mark.parametrize("d,dtype", [(64, H), (128, F)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
@pytest.mark.parametrize("causal", [False, True])
def test_any_negative_id_is_padding(d, dtype, cap, bias, causal):
    # (also in the middle, and as whole warps of rows beside rows of documents)
    for lengths, pad in (([150, 100], 70), ([60, 3, 200, 90], 7), ([60, 100], 96), ([20, 50, 80], 200)):
        dq = docs_of(lengths, pad, 2)
        dq[1, 40:55] = -1
        one = check(2, 2, 1, dq.shape[1], dq.shape[1], d, dtype, causal=causal, cap=cap, bias=bias, dq=dq)
        for other in (-2, -7, -2 ** 31):
            ids = torch.where(dq < 0, torch.full_like(dq, other), dq)
            same = check(2, 2, 1, dq.shape[1], dq.shape[1], d, dtype, causal=causal, cap=cap, bias=bias, dq=ids)
            assert all(torch.equal(x, y) for x, y in zip(one, same))
            assert (same[1][1, :, 40:55] == -math.inf).all()


def test_keys_ahead_may_be_infinite_scores():
    # a masked key whose score is infinite or NaN leaves the rows that do not see it alone
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, 1, 256, 64, generator=g).half() for _ in "qkv")
    k2 = k.clone()
    k2[:, :, 200] = math.nan
    k2[:, :, 220] = math.inf
    import quantized_attention_mean_gb300 as qa
    a = qa.scored_attn(q.to(DEV), k.to(DEV), v.to(DEV), is_causal=True, softcap=20.0)
    b = qa.scored_attn(q.to(DEV), k2.to(DEV), v.to(DEV), is_causal=True, softcap=20.0)
    assert torch.equal(a[:, :, :200], b[:, :, :200]) and torch.isnan(b[:, :, 200:]).any()


@pytest.mark.parametrize("d,dtype", [(64, H), (64, F), (128, H), (128, F)])
@pytest.mark.parametrize("bias", [False, True])
def test_keys_no_row_of_a_warp_sees_leave_the_capped_scores_alone(d, dtype, bias):
    # large finite scores of keys that are padding, lie behind the last one seen, or are of documents that only other
    # warps' rows see: the other rows stay as they are, bit for bit (fp32 statistics with them)
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(12)
    n = 256
    q, k, v = (torch.randn(1, 2, n, d, generator=g).to(dtype) for _ in "qkv")
    slopes = torch.tensor([0.02, 0.01], device=DEV) if bias else None
    ids_k = (torch.arange(n, dtype=torch.int32) % 2)[None].contiguous()
    ids_q = (torch.arange(n, dtype=torch.int32) // 128)[None].contiguous()
    pad = torch.zeros(1, n, dtype=torch.int32)
    pad[0, 5::9] = -1
    cases = [(dict(doc_ids=ids_q, doc_ids_k=ids_k), torch.arange(1, n, 2), slice(0, 128)),     # (the first 128 rows: even keys)
             (dict(doc_ids=pad, is_causal=True), torch.arange(5, n, 9), slice(0, n)),
             (dict(is_causal=True, q_offset=-41), torch.arange(n - 41, n), slice(0, n))]
    for kw, unseen, rows in cases:
        kw = {x: y.to(DEV) if torch.is_tensor(y) else y for x, y in kw.items()}
        got = []
        for size in (1.0, 100.0, 30000.0):
            kk, qq = k.clone(), q.clone()
            kk[:, :, unseen] = (q[:, :, unseen] * size).clamp(-60000, 60000)
            if "is_causal" in kw and "doc_ids" in kw:
                qq[:, :, unseen] = kk[:, :, unseen]                       # (rows that are padding)
            got.append(qa.scored_attn(qq.to(DEV), kk.to(DEV), v.to(DEV), softcap=25.0, slopes=slopes, return_lse=True, **kw))
        for out, lse in got[1:]:
            assert torch.equal(out[:, :, rows], got[0][0][:, :, rows])
            assert torch.equal(lse[:, :, rows], got[0][1][:, :, rows])


@pytest.mark.parametrize("nq,nk,offset,prefix", [(100, 300, 50, None), (300, 700, 77, None), (5, 4000, 2100, None),
                                                 (100, 300, 0, [170]), (260, 300, -20, None)])
@pytest.mark.parametrize("d,dtype", [(64, H), (128, F)])
@pytest.mark.parametrize("bias", [False, True])
def test_keys_behind_the_last_seen_may_hold_anything(nq, nk, offset, prefix, d, dtype, bias):
    # a buffer longer than the tokens it holds: the rest of the last tile is garbage
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(1, 1, nk, d, generator=g).to(dtype) for _ in "kv")
    held = max(nq + offset, *(prefix or [0]))
    clean = v.clone()
    clean[:, :, held:] = 0
    k[:, :, held:], v[:, :, held::2], v[:, :, held + 1::2] = math.nan, math.nan, -math.inf
    check(1, 2, 1, nq, nk, d, dtype, causal=True, offset=offset, prefix=prefix, bias=bias, k=k, v=v, clean=clean)


def test_large_scores_and_growing_maximum():
    # scores rise along the keys by far more than the frame allows, then fall
    n, d = 700, 64
    k = torch.zeros(1, 1, n, d)
    k[0, 0, :, 0] = torch.cat([torch.linspace(-60, 60, 500), torch.linspace(60, -200, 200)])
    q = torch.ones(1, 1, 130, d)
    v = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1))
    check(1, 1, 1, 130, n, d, F, q=q.half(), k=k.half(), v=v.half(), scale=1.0)
    check(1, 1, 1, 130, n, d, H, q=q.bfloat16(), k=k.bfloat16(), v=v.bfloat16(), scale=1.0, bias=True)
    check(1, 1, 1, 130, n, d, F, q=q.half(), k=k.half(), v=v.half(), scale=1.0, cap=50.0, causal=True, offset=n)


@pytest.mark.parametrize("cap,relative", [(1000.0, True), (4096.0, False), (1.0, False), (1e-3, False)])
def test_caps_from_tiny_to_large(cap, relative):
    for d, dtype in ((64, F), (128, H)):
        check(1, 2, 1, 300, 300, d, dtype, cap=cap, relative_cap=relative)
        check(1, 2, 1, 300, 300, d, dtype, cap=cap, causal=True, bias=True, relative_cap=relative)


def test_slopes_of_either_sign():
    # a negative slope favours distant keys: the maximum moves with every tile
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(8)
    for d, dtype in ((64, F), (128, H)):
        q, k, v = (torch.randn(1, 4, 600, d, generator=g).to(dtype) for _ in "qkv")
        slopes = torch.tensor([-0.3, -0.01, 0.0, 2.0])
        dist = (torch.arange(600)[:, None] - torch.arange(600)).abs().double()
        b = (-slopes.double()[:, None, None] * dist)[None].to(DEV)
        for causal in (False, True):
            out, lse = qa.scored_attn(*(t.to(DEV) for t in (q, k, v)), is_causal=causal, slopes=slopes.to(DEV), return_lse=True)
            seen = visible(600, 600, 1, causal, 0, None, None, None)[:, None].expand(1, 4, 600, 600).to(DEV)
            r = attend(*(t.to(DEV) for t in (q, k, v)), d ** -0.5, 0.0, b, seen, dtype)
            assert_close(out, r["out"], r["out_tol"], "out")
            assert_close(lse, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("d,dtype", [(64, H), (128, F)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_offsets_near_the_ends_of_32_bits(d, dtype, cap):
    for offset in (-0x7fffff00 + 40000, 0x7fffff00 - 4, -40000, 2 ** 24 + 1):
        check_slopes(d, dtype, cap, offset)
    # a distance that passes 2^31 is refused; without slopes there is none
    import quantized_attention_mean_gb300 as qa
    q, k = (torch.randn(1, 1, n, d, device=DEV).to(dtype) for n in (4, 300))
    for offset in (-0x7fffff00, -0x7fffff00 + 299):
        with pytest.raises(qa.SageError):
            qa.scored_attn(q, k, k, slopes=torch.ones(1, device=DEV), q_offset=offset, softcap=cap)
        assert torch.equal(qa.scored_attn(q, k, k, q_offset=offset, softcap=cap), qa.scored_attn(q, k, k, softcap=cap))


def check_slopes(d, dtype, cap, offset):
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(13)
    nq, nk = 4, 40000
    q, k, v = (torch.randn(1, h, n, d, generator=g).to(dtype).to(DEV) for h, n in ((2, nq), (1, nk), (1, nk)))
    slopes = torch.tensor([1e-3, -2e-4])
    dist = (torch.arange(nq)[:, None] + offset - torch.arange(nk)).abs().double()
    b = (-slopes.double()[:, None, None] * dist)[None].to(DEV)
    out, lse = qa.scored_attn(q, k, v, slopes=slopes.to(DEV), q_offset=offset, softcap=cap, return_lse=True)
    kk, vv = (t.expand(1, 2, nk, d) for t in (k, v))
    r = attend(q, kk, vv, d ** -0.5, cap, b, dtype=dtype)
    assert_close(out, r["out"], r["out_tol"], f"out at {offset}")
    assert_close(lse, r["lse"], r["lse_tol"], f"lse at {offset}")


def test_strided_and_broadcast_inputs():
    g = torch.Generator().manual_seed(6)
    # a fused projection's slices: rows of one tensor
    B, n, h, d = 2, 200, 3, 64
    qkv = torch.randn(B, n, 3, h, d, generator=g).bfloat16()
    q, k, v = (qkv[:, :, i] for i in range(3))
    fused = qkv.to(DEV)
    order = iter(range(3))
    check(B, h, h, n, n, d, H, "NHD", causal=True, q=q.transpose(1, 2), k=k.transpose(1, 2), v=v.transpose(1, 2),
          place=lambda t: fused[:, :, next(order)])
    # keys and values shared over the batch by a zero stride, rows that start at odd elements
    k1, v1 = (torch.randn(1, 2, 300, 64, generator=g).half() for _ in "kv")
    k2, v2 = k1.expand(2, -1, -1, -1), v1.expand(2, -1, -1, -1)
    q = torch.randn(2, 2, 100, 64, generator=g).half()

    def odd(t):
        if t.shape[2] == 300:
            return t[:1].to(DEV).expand(2, -1, -1, -1)
        w = torch.zeros(2, 2, 100, 67, dtype=torch.float16, device=DEV)
        w[..., 1:65] = t.to(DEV)
        return w[..., 1:65]
    check(2, 2, 2, 100, 300, 64, F, q=q, k=k2, v=v2, place=odd)


def test_without_a_workspace():
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(2, 4, 300, 64, generator=g).half().to(DEV) for _ in "qkv")
    n = qa.scored_attn_workspace_bytes(2, 4, 4, 300, 300, 64, documents=False)
    assert n == 256
    ws = qa.alloc_workspace(n, DEV)
    ws.fill_(255)
    a = qa.scored_attn(q, k, v, is_causal=True, softcap=20.0, workspace=ws)
    assert qa.read_device_status(ws) == 0
    assert torch.equal(qa.scored_attn(q, k, v, is_causal=True, softcap=20.0), a)
    assert torch.equal(qa.scored_attn(q[:, :, :0], k, v), q[:, :, :0])
    assert (qa.scored_attn(q, k[:, :, :0], v[:, :, :0]) == 0).all()


def test_no_keys_and_out_strides():
    import quantized_attention_mean_gb300 as qa
    q = torch.randn(1, 2, 5, 64, dtype=torch.float16, device=DEV)
    e = torch.empty(1, 2, 0, 64, dtype=torch.float16, device=DEV)
    out, lse = qa.scored_attn(q, e, e, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert qa.scored_attn(q[:, :, :0], q, q).shape == (1, 2, 0, 64)
    k = torch.randn(1, 2, 300, 64, dtype=torch.float16, device=DEV)
    want = qa.scored_attn(q, k, k)
    for width, at in ((67, 1), (80, 8)):
        wide = torch.full((1, 2, 5, width), 7.0, dtype=torch.float16, device=DEV)
        qa.scored_attn(q, k, k, out=wide[..., at:at + 64])
        assert torch.equal(wide[..., at:at + 64], want)
        assert (wide[..., :at] == 7).all() and (wide[..., at + 64:] == 7).all()


def test_no_rows_no_keys_no_sequences():
    import quantized_attention_mean_gb300 as qa
    q, k = (torch.randn(2, 2, n, 64, dtype=torch.float16, device=DEV) for n in (5, 130))
    ids = lambda n: torch.zeros(2, n, dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = qa.scored_attn(q, k[:, :, :0], k[:, :, :0], doc_ids=ids(5), doc_ids_k=ids(0), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert qa.scored_attn(q[:, :, :0], k, k, doc_ids=ids(0), doc_ids_k=ids(130)).shape == (2, 2, 0, 64)
    assert qa.scored_attn(q[:, :, :0], k[:, :, :0], k[:, :, :0], doc_ids=ids(0)).shape == (2, 2, 0, 64)
    for rows, keys in ((q[:, :, :0], k), (q[:, :, :0], k[:, :, :0]), (q[:0], k[:0]), (q[:0, :, :0], k[:0, :, :0])):
        out, lse = qa.scored_attn(rows, keys, keys, is_causal=True, return_lse=True)
        assert out.shape == rows.shape and lse.shape == rows.shape[:3]
    assert qa.scored_attn(q[:0], k[:0], k[:0], doc_ids=ids(5)[:0], doc_ids_k=ids(130)[:0]).shape == (0, 2, 5, 64)


def test_in_a_graph_and_on_another_stream():
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(1, 4, 300, 128, generator=g).bfloat16().to(DEV) for _ in "qkv")
    ids = docs_of([100, 180], 20, 1).to(DEV)
    kw = dict(is_causal=True, softcap=30.0, doc_ids=ids)
    eager = qa.scored_attn(q, k, v, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = qa.scored_attn(q, k, v, stream=side, **kw)
    side.synchronize()
    assert torch.equal(other, eager)
    ws = qa.alloc_workspace(qa.scored_attn_workspace_bytes(1, 4, 4, 300, 300, 128), DEV)
    out = torch.empty_like(q)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:                                  # two graphs over one workspace
        with torch.cuda.graph(gr):
            qa.scored_attn(q, k, v, out=out, workspace=ws, **kw)
    for gr in graphs * 2:
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_captured_without_a_workspace():
    # what a captured call takes from the allocator must not be what a later one of the graph is given while it runs
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, h, n, 64, generator=g).half().to(DEV) for h, n in ((4, 200), (2, 9000), (2, 9000)))
    ids = torch.randint(0, 3, (1, 9000), generator=g, dtype=torch.int32).to(DEV)
    cache = [t[0].transpose(0, 1).reshape(1, 9000, 2, 64)[:, :8960].reshape(560, 16, 2, 64).contiguous() for t in (k, v)]
    table, lens = torch.arange(560, dtype=torch.int32, device=DEV)[None], torch.tensor([8960], dtype=torch.int32, device=DEV)
    mass0 = torch.rand(560, 2, 16, generator=g).to(DEV)
    pos = torch.arange(16, dtype=torch.int32, device=DEV).expand(560, 2, 16).contiguous()

    def step(c, mass, pos):
        a = qa.scored_attn(q, k, v, is_causal=True, q_offset=8800, doc_ids=ids[:, :200].contiguous(), doc_ids_k=ids)
        b = qa.paged_attn(a[:, :, 7], *c, table, lens, 10 ** 5, tensor_layout="NHD", mass=mass)
        n = qa.paged_evict(*c, mass, pos, table, lens, 500, 9000, tensor_layout="NHD")
        d = qa.scored_attn(q * 0.5, k, v)
        return a, b, n, d, mass, pos, *c

    want = step([t.clone() for t in cache], mass0.clone(), pos.clone())
    graph, side = torch.cuda.CUDAGraph(), [t.clone() for t in (*cache, mass0, pos)]
    with torch.cuda.graph(graph):
        got = step([side[0], side[1]], side[2], side[3])
    for _ in range(3):
        for t, x in zip(side, (*cache, mass0, pos)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_prompt_in_chunks_then_decode():
    """A prompt attended in two chunks, its keys appended to a paged cache, then one more token from
    the cache: the same rows as one call over the whole."""
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(9)
    n, hq, hkv, d, page = 401, 4, 2, 64, 16
    q, k, v = (torch.randn(1, n, h, d, generator=g).half().to(DEV) for h in (hq, hkv, hkv))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0], device=DEV)
    kw = dict(tensor_layout="NHD", is_causal=True, softcap=25.0, slopes=slopes, return_lse=True)
    whole, lse = qa.scored_attn(q, k, v, **kw)
    first, l1 = qa.scored_attn(q[:, :250], k[:, :250], v[:, :250], **kw)
    second, l2 = qa.scored_attn(q[:, 250:400], k[:, :400], v[:, :400], q_offset=250, **kw)
    cache = [torch.zeros(30, hkv, page, d, dtype=torch.float16, device=DEV) for _ in "kv"]
    table = torch.randperm(30, generator=g)[None, :26].to(torch.int32).to(DEV).contiguous()
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    qa.paged_append(k[0], v[0], *cache, table, lens, cu_seqlens=cu)
    last, l3 = qa.paged_attn(q[:, 400], *cache, table, lens + n, 416, softcap=25.0, slopes=slopes, return_lse=True)
    # both sides round once from nearly equal values: at most one step of fp16 apart, relative 2^-10
    got = torch.cat([first, second, last[:, None]], 1).float()
    assert ((got - whole.float()).abs() <= 2.0 ** -10 * whole.float().abs() + 2.0 ** -10).all()
    assert ((torch.cat([l1, l2, l3[..., None]], 2) - lse).abs() <= 1e-4).all()
