"""Decode attention over a paged cache, appending to it and evicting from it, against float64 and
plain loops."""

import math
import os
import textwrap
import types

import pytest
import torch

import paged_reference as ref
from attn_reference import assert_close, attend

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def on_gpu(c):
    return {n: (t.to(DEV) if torch.is_tensor(t) else t) for n, t in c.items()}


def decode_reference(c, q, sm_scale, cap=0.0, slopes=None, kpos=None, qpos=None, hkv=1):
    B, hq, d = q.shape
    g = hq // hkv
    res = dict(out=torch.zeros(B, hq, d, dtype=torch.float64), lse=torch.full((B, hq), -math.inf, dtype=torch.float64),
               out_tol=torch.zeros(B, hq, d, dtype=torch.float64), lse_tol=torch.ones(B, hq, dtype=torch.float64), p={}, p_tol={})
    for b, n in enumerate(c["lens"].tolist()):
        if n == 0:
            continue
        for h in range(hkv):
            bias = None
            if slopes is not None:
                p, s = ref.place(c, b, n)
                where = torch.arange(n) if kpos is None else kpos[p, h, s]
                at = n - 1 if qpos is None else int(qpos[b])
                bias = -slopes[h * g:(h + 1) * g, None].double() * (at - where.double()).abs()
            r = attend(q[b, h * g:(h + 1) * g], ref.rows(c, "k", b, h, n), ref.rows(c, "v", b, h, n), sm_scale, cap, bias,
                       dtype=q.dtype)
            for name in ("out", "lse", "out_tol", "lse_tol"):
                res[name][b, h * g:(h + 1) * g] = r[name]
            res["p"][b, h], res["p_tol"][b, h] = r["p"].sum(0), r["p_tol"].sum(0)
    return res


CASES = [
    # lens, hq, hkv, d, page, dtype, layout, cap, slopes
    ([1], 1, 1, 64, 16, torch.float16, "HND", 0.0, False),
    ([1, 0, 17, 64, 65], 8, 2, 128, 16, torch.bfloat16, "HND", 0.0, False),
    ([300, 5, 0, 129], 14, 2, 128, 7, torch.bfloat16, "NHD", 30.0, False),      # group of 7, pages of 7
    ([63, 2000, 1], 16, 1, 64, 48, torch.float16, "NHD", 0.0, True),
    ([500, 777], 40, 2, 72, 32, torch.float16, "HND", 20.0, True),              # group of 20: two row blocks
    ([130, 1, 90], 6, 3, 33, 8, torch.bfloat16, "HND", 0.0, False),             # rows no 16-byte load fits
    ([4097] * 3, 32, 8, 128, 64, torch.bfloat16, "HND", 0.0, False),
    ([20001], 8, 8, 96, 128, torch.bfloat16, "NHD", 50.0, True),                # one sequence over many CTAs
    ([3] * 150, 4, 4, 64, 4, torch.float16, "HND", 0.0, False),                 # more sequences than threads scan at once
    ([0, 0], 4, 2, 64, 16, torch.float16, "HND", 0.0, False),
]


# (a bound far above the lengths takes the form for long sequences)
@pytest.mark.parametrize("bound", [0, 10 ** 5])
@pytest.mark.parametrize("lens,hq,hkv,d,page,dtype,layout,cap,biased", CASES)
def test_decode(lens, hq, hkv, d, page, dtype, layout, cap, biased, bound):
    import quantized_attention_mean_gb300 as qa
    bound = max(max(lens), bound)
    c = ref.make_cache(lens, hkv, d, page, dtype, layout, seed=len(lens) + d)
    g = torch.Generator().manual_seed(5)
    q = (torch.randn(len(lens), hq, d, generator=g) * 2).to(dtype)
    slopes = 2.0 ** (-torch.arange(1, hq + 1).float() / 4) if biased else None
    G = on_gpu(c)
    ws = qa.alloc_workspace(qa.paged_attn_workspace_bytes(len(lens), hq, hkv, bound, d), DEV)
    ws.fill_(255)
    out, lse = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], bound, tensor_layout=layout,
                             softcap=cap, slopes=None if slopes is None else slopes.to(DEV), return_lse=True, workspace=ws)
    assert qa.read_device_status(ws) == 0
    r = decode_reference(c, q, 1 / math.sqrt(d), cap, slopes, hkv=hkv)
    assert_close(out, r["out"], r["out_tol"] + 1e-12, "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")


def test_decode_positions_strides_and_scale():
    # explicit positions in an order of their own, a cache that is a slice of a wider one, strided q and out
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([200, 33], 2, 64, 16, torch.float16, "HND")
    hkv, d, hq = 2, 64, 8
    g = torch.Generator().manual_seed(1)
    kpos = torch.randint(0, 5000, (c["k"].shape[0], hkv, 16), generator=g, dtype=torch.int32)
    qpos = torch.tensor([5001, 77], dtype=torch.int32)
    q = torch.randn(2, hq, d, generator=g).half()
    slopes = torch.linspace(0.001, 0.02, hq)
    G = on_gpu(c)
    wide = torch.zeros(c["k"].shape[0], hkv, 16, 2 * d + 8, dtype=torch.float16, device=DEV)
    wide[..., 8:8 + d], wide[..., 8 + d:] = G["k"], G["v"]
    qw = torch.zeros(2, 2 * hq, d, dtype=torch.float16, device=DEV)
    qw[:, ::2] = q.to(DEV)
    ow = torch.full((2, 2 * hq, d), 9.0, dtype=torch.float16, device=DEV)
    lse = torch.empty(2, hq, device=DEV)
    qa.paged_attn(qw[:, ::2], wide[..., 8:8 + d], wide[..., 8 + d:], G["table"], G["lens"], 999, sm_scale=0.3,
                  slopes=slopes.to(DEV), key_positions=kpos.to(DEV), q_positions=qpos.to(DEV), return_lse=True,
                  out=ow[:, ::2], lse=lse)
    r = decode_reference(c, q, 0.3, 0.0, slopes, kpos, qpos, hkv)
    assert_close(ow[:, ::2], r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")
    assert (ow[:, 1::2] == 9).all()


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("planes", [False, True])
def test_decode_positions_near_the_ends_of_32_bits(d, dtype, planes):
    # the distance from the query's position to a slot passes 2^31
    import quantized_attention_mean_gb300 as qa
    n = 40000
    c = ref.make_cache([n], 1, d, 64, dtype)
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    slopes = torch.tensor([1e-3, -2e-4, 1e-4, 0.0])
    kpos = None
    if planes:
        kpos = torch.zeros(c["k"].shape[0], 1, 64, dtype=torch.int32)
        p, s = ref.place(c, 0, n)
        kpos[p, 0, s] = torch.arange(n, dtype=torch.int32)
    G = on_gpu(c)
    for at in (-2 ** 31, -2 ** 31 + n // 2, 2 ** 31 - 1):
        qpos = torch.tensor([at], dtype=torch.int32)
        out, lse = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], n, slopes=slopes.to(DEV),
                                 key_positions=None if kpos is None else kpos.to(DEV), q_positions=qpos.to(DEV), return_lse=True)
        r = decode_reference(c, q, d ** -0.5, 0.0, slopes, kpos, qpos.long(), 1)
        assert_close(out, r["out"], r["out_tol"], f"out at {at}")
        assert_close(lse, r["lse"], r["lse_tol"], f"lse at {at}")


@pytest.mark.parametrize("bound", [700, 9000])
@pytest.mark.parametrize("hq,hkv,d,cap", [(8, 2, 128, 0.0), (20, 1, 64, 30.0), (3, 3, 40, 0.0)])
def test_decode_accumulates_weights(hq, hkv, d, cap, bound):
    import quantized_attention_mean_gb300 as qa
    lens = [700, 1, 0, 65]
    c = ref.make_cache(lens, hkv, d, 16, torch.bfloat16)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(4, hq, d, generator=g).bfloat16()
    mass0 = torch.rand(c["k"].shape[0], hkv, 16, generator=g)
    G, mass = on_gpu(c), mass0.to(DEV)
    for _ in range(2):
        qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], bound, softcap=cap, mass=mass)
    r = decode_reference(c, q, 1 / math.sqrt(d), cap, hkv=hkv)
    want, tol = mass0.double(), mass0.double() * 2.0 ** -22 + 1e-7
    for (b, h), p in r["p"].items():
        at, s = ref.place(c, b, lens[b])
        want[at, h, s] += 2 * p
        tol[at, h, s] += 2 * r["p_tol"][b, h] + 2 * p * 2.0 ** -22
    assert_close(mass, want, tol, "mass")


def test_decode_mass_of_shared_and_odd_pages():
    # a prompt's pages shared by three sequences, pages of six slots, positions of their own for the bias
    import quantized_attention_mean_gb300 as qa
    hq, hkv, d, page = 4, 2, 64, 6
    c = ref.make_cache([100, 100, 100], hkv, d, page, torch.float16, seed=2)
    c["table"][1, :8] = c["table"][0, :8]
    c["table"][2, :8] = c["table"][0, :8]
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, hq, d, generator=g).half()
    kpos = torch.randint(0, 200, (c["k"].shape[0], hkv, page), generator=g, dtype=torch.int32)
    qpos = torch.tensor([200, 210, 300], dtype=torch.int32)
    slopes = torch.tensor([0.01, 0.02, -0.01, 0.0])
    G, mass = on_gpu(c), torch.zeros(c["k"].shape[0], hkv, page, device=DEV)
    out = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], 100, slopes=slopes.to(DEV),
                        key_positions=kpos.to(DEV), q_positions=qpos.to(DEV), mass=mass)
    r = decode_reference(c, q, d ** -0.5, 0.0, slopes, kpos, qpos, hkv)
    assert_close(out, r["out"], r["out_tol"], "out")
    want = torch.zeros(mass.shape, dtype=torch.float64)
    tol = want + 1e-7
    for (b, h), p in r["p"].items():
        at, s = ref.place(c, b, 100)
        want[at, h, s] += p
        tol[at, h, s] += r["p_tol"][b, h] + 3 * 2.0 ** -23       # sums of up to six, each below 8: two additions
    assert_close(mass, want, tol, "mass")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 24])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_decode_pages_of_eight_row_blocks(d, page, layout):
    import quantized_attention_mean_gb300 as qa
    lens = [1, 8, 9, 23, 24, 25, 500]
    c = ref.make_cache(lens, 2, d, page, torch.bfloat16, layout, seed=d + page)
    q = torch.randn(len(lens), 6, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    G = on_gpu(c)
    for bound in (500, 10 ** 5):
        out = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], bound, tensor_layout=layout)
        r = decode_reference(c, q, d ** -0.5, hkv=2)
        assert_close(out, r["out"], r["out_tol"], "out")


def test_empty_cache_in_place_and_from_another_page():
    import quantized_attention_mean_gb300 as qa
    # a cache without pages
    k = torch.empty(0, 2, 16, 64, dtype=torch.float16, device=DEV)
    table, lens = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    q = torch.randn(2, 4, 64, dtype=torch.float16, device=DEV)
    for bound in (0, 10 ** 5):
        out, lse = qa.paged_attn(q, k, k, table, lens, bound, return_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    # the output over the query
    c = ref.make_cache([300, 40], 2, 64, 16, torch.float16, room=16)
    G = on_gpu(c)
    for bound in (300, 10 ** 5):
        want = qa.paged_attn(q, G["k"], G["v"], G["table"], G["lens"], bound)
        both = q.clone()
        qa.paged_attn(both, G["k"], G["v"], G["table"], G["lens"], bound, out=both)
        assert torch.equal(both, want)
    # a sequence's first page appended to both, as a shared prefix is copied
    page = int(c["table"][0, 0])
    src = [G[n][page].transpose(0, 1).repeat(2, 1, 1) for n in "kv"]
    view = [G[n][page].transpose(0, 1) for n in "kv"]
    cu = torch.tensor([0, 16, 32], dtype=torch.int32, device=DEV)
    other = [G[n].clone() for n in "kv"]
    qa.paged_append(*src, *other, G["table"], G["lens"], cu_seqlens=cu)
    one = torch.tensor([0, 16, 16], dtype=torch.int32, device=DEV)
    two = torch.tensor([0, 0, 16], dtype=torch.int32, device=DEV)
    qa.paged_append(*view, G["k"], G["v"], G["table"], G["lens"], cu_seqlens=one)
    qa.paged_append(*view, G["k"], G["v"], G["table"], G["lens"], cu_seqlens=two)
    assert torch.equal(G["k"], other[0]) and torch.equal(G["v"], other[1])


@pytest.mark.parametrize("page,d", [(16, 64), (4, 128), (16, 33)])
def test_without_a_workspace(page, d):
    # (pages by TMA, by 16 bytes and element by element; an output row that starts anywhere)
    import quantized_attention_mean_gb300 as qa
    lens = [300, 1, 77]
    c = ref.make_cache(lens, 2, d, page, torch.float16)
    G = on_gpu(c)
    q = torch.randn(3, 6, d + 1, generator=torch.Generator().manual_seed(2)).half()[..., 1:]
    ws = qa.alloc_workspace(qa.paged_attn_workspace_bytes(3, 6, 2, 300, d), DEV)
    assert ws.numel() == 256
    wide = torch.zeros(3, 6, d + 1, dtype=torch.float16, device=DEV)
    wide[..., 1:] = q.to(DEV)
    a = qa.paged_attn(wide[..., 1:], G["k"], G["v"], G["table"], G["lens"], 300, workspace=ws)
    b = qa.paged_attn(wide[..., 1:], G["k"], G["v"], G["table"], G["lens"], 300)
    assert qa.read_device_status(ws) == 0 and torch.equal(a, b)
    r = decode_reference(c, q, d ** -0.5, hkv=2)
    assert_close(b, r["out"], r["out_tol"], "out")
    table = G["table"].clone()
    table[0, 1] = c["k"].shape[0]
    qa.paged_attn(wide[..., 1:], G["k"], G["v"], table, G["lens"], 300)           # a bad page: zeros, and no word of it
    qa.paged_attn(wide[..., 1:], G["k"], G["v"], table, G["lens"], 300, workspace=ws)
    assert qa.read_device_status(ws) == 13


def test_append_and_evict_in_a_graph():
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([70, 20], 2, 64, 16, torch.float16, room=2)
    shape = (c["k"].shape[0], 2, 16)
    mass0 = torch.rand(shape, device=DEV)
    pos0 = torch.zeros(shape, dtype=torch.int32, device=DEV)
    k = torch.randn(2, 2, 64, dtype=torch.float16, device=DEV)
    ws = qa.alloc_workspace(qa.paged_evict_workspace_bytes(2, 2, 80, 32), DEV)

    def state():
        G = on_gpu(c)
        return [G["k"], G["v"], mass0.clone(), pos0.clone(), G["table"], G["lens"]]

    def step(s):
        qa.paged_append(k, k, s[0], s[1], s[4], s[5], mass=s[2], key_positions=s[3])
        return qa.paged_evict(s[0], s[1], s[2], s[3], s[4], s[5] + 1, 32, 80, recent=8, workspace=ws)

    eager, s = state(), state()
    want = step(eager)
    first = [t.clone() for t in s]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = step(s)
    for _ in range(2):
        for t, f in zip(s, first):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(new, want) and all(torch.equal(x, y) for x, y in zip(s, eager))


def test_a_cache_past_32_bits():
    # pages whose rows lie more than 2^32 elements into the cache
    import quantized_attention_mean_gb300 as qa
    pages, hkv, page, d = 300000, 1, 128, 128                    # 9.8 GB each
    k = torch.empty(pages, hkv, page, d, dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    mass = torch.zeros(pages, hkv, page, device=DEV)
    pos = torch.zeros(pages, hkv, page, dtype=torch.int32, device=DEV)
    at = torch.tensor([299999, 1, 299998, 270000], dtype=torch.int32)
    small = ref.make_cache([400], hkv, d, page, torch.float16, spare=0)
    small["table"][0] = torch.arange(4, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(400, hkv, d, generator=g).half() for _ in "kv"]
    table, lens = at[None].to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 400], dtype=torch.int32, device=DEV)
    qa.paged_append(*(t.to(DEV) for t in new), k, v, table, lens, cu_seqlens=cu, mass=mass, key_positions=pos)
    p, s = ref.place(small, 0, 400)
    for which, t in zip("kv", new):
        small[which][p, :, s] = t
    q = torch.randn(1, 4, d, generator=g).half()
    out = qa.paged_attn(q.to(DEV), k, v, table, lens + 400, 400, mass=mass)
    r = decode_reference(small, q, d ** -0.5, hkv=hkv)
    assert_close(out, r["out"], r["out_tol"], "out")
    held = at.long().to(DEV)
    few, fp = mass[held].cpu(), pos[held].cpu()
    qa.paged_evict(k, v, mass, pos, table, lens + 400, 100, 400, recent=10)
    ref.evict(small, few, fp, 100, 0, 10)
    assert torch.equal(mass[held].cpu(), few) and torch.equal(pos[held].cpu(), fp)
    keep, ks = ref.place(small, 0, 100)
    assert torch.equal(k[held].cpu()[keep, :, ks], small["k"][keep, :, ks])
    assert torch.equal(v[held].cpu()[keep, :, ks], small["v"][keep, :, ks])


def test_decode_masked_garbage_and_nan():
    # slots behind a sequence's end and unused pages hold NaN: nothing of them may show
    import quantized_attention_mean_gb300 as qa
    lens = [70, 5]
    c = ref.make_cache(lens, 2, 128, 16, torch.bfloat16)
    clean = {n: t.clone() if torch.is_tensor(t) else t for n, t in c.items()}
    used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        p, s = ref.place(c, b, n)
        used[p, s] = True
    for w in "kv":
        c[w][(~used)[:, None, :].expand(-1, 2, -1)] = math.nan
    q = torch.randn(2, 8, 128).bfloat16()
    G = on_gpu(c)
    out = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], G["lens"], 70)
    r = decode_reference(clean, q, 1 / math.sqrt(128), hkv=2)
    assert_close(out, r["out"], r["out_tol"], "out")


@pytest.mark.parametrize("bound", [40, 9000])
def test_decode_reports_bad_lengths_and_pages(bound):
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([40, 40, 40], 2, 64, 16, torch.float16)
    q = torch.randn(3, 4, 64).half().to(DEV)
    G = on_gpu(c)
    ws = qa.alloc_workspace(qa.paged_attn_workspace_bytes(3, 4, 2, bound, 64), DEV)
    good = qa.paged_attn(q, G["k"], G["v"], G["table"], G["lens"], bound, workspace=ws)
    assert qa.read_device_status(ws) == 0
    for bad in (-1, 49, 2 ** 31 - 1) + ((41,) if bound == 40 else ()):     # (three pages hold 48)
        lens = G["lens"].clone()
        lens[1] = bad
        out, lse = qa.paged_attn(q, G["k"], G["v"], G["table"], lens, bound, workspace=ws, return_lse=True)
        assert qa.read_device_status(ws) == 12
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    for bad in (-1, c["k"].shape[0], 2 ** 31 - 1):
        table = G["table"].clone()
        table[2, 1] = bad
        out = qa.paged_attn(q, G["k"], G["v"], table, G["lens"], bound, workspace=ws)
        assert qa.read_device_status(ws) == 13
        assert torch.equal(out[:2], good[:2]) and torch.isfinite(out).all()
    qa.paged_attn(q, G["k"], G["v"], G["table"], G["lens"], bound, workspace=ws)
    assert qa.read_device_status(ws) == 0


APPENDS = [
    # old lengths, new counts (None: one each), hkv, d, page, dtype, layout
    ([0, 15, 16, 100], None, 8, 128, 16, torch.bfloat16, "HND"),
    ([3, 0, 50], [5, 0, 130], 2, 64, 7, torch.float16, "NHD"),
    ([10, 2], [1, 33], 3, 35, 8, torch.bfloat16, "NHD"),
    ([0], [1000], 1, 80, 64, torch.float16, "HND"),
]


@pytest.mark.parametrize("old,new,hkv,d,page,dtype,layout", APPENDS)
@pytest.mark.parametrize("planes", [False, True])
def test_append(old, new, hkv, d, page, dtype, layout, planes):
    import quantized_attention_mean_gb300 as qa
    counts = [1] * len(old) if new is None else new
    tail = 0 if new is None else 3                      # tokens behind the last sequence
    c = ref.make_cache(old, hkv, d, page, dtype, layout, room=max(counts))
    g = torch.Generator().manual_seed(3)
    T = sum(counts) + tail
    k, v = (torch.randn(T, hkv, d, generator=g).to(dtype) for _ in "kv")
    cu = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
    mass = torch.full((c["k"].shape[0], hkv, page), 5.0) if planes else None
    kpos = torch.full((c["k"].shape[0], hkv, page), -3, dtype=torch.int32) if planes else None
    pos = torch.randint(0, 9999, (T,), generator=g, dtype=torch.int32) if planes else None
    G = on_gpu(c)
    gm, gp, gpos = (None if t is None else t.to(DEV) for t in (mass, kpos, pos))
    ws = qa.alloc_workspace(256, DEV)
    qa.paged_append(k.to(DEV), v.to(DEV), G["k"], G["v"], G["table"], G["lens"],
                    cu_seqlens=None if new is None else cu.to(DEV), tensor_layout=layout, mass=gm, key_positions=gp,
                    positions=gpos, workspace=ws)
    assert qa.read_device_status(ws) == 0
    t = 0
    for b, n in enumerate(counts):
        p, s = ref.place(c, b, old[b] + n)
        for i in range(old[b], old[b] + n):
            for h in range(hkv):
                ref.set_row(c, "k", p[i], h, s[i], k[t, h])
                ref.set_row(c, "v", p[i], h, s[i], v[t, h])
                if planes:
                    mass[p[i], h, s[i]] = 0.0
                    kpos[p[i], h, s[i]] = pos[t]
            t += 1
    assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])
    if planes:
        assert torch.equal(gm.cpu(), mass) and torch.equal(gp.cpu(), kpos)


def test_calls_with_nothing_to_do_clear_the_status():
    # a workspace that held another call's error
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([30, 5], 2, 64, 16, torch.float16)
    G = on_gpu(c)
    table, lens = G["table"][:0], G["lens"][:0]
    x = torch.randn(2, 2, 64, dtype=torch.float16, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    mass, pos = torch.zeros(c["k"].shape[0], 2, 16, device=DEV), torch.zeros(c["k"].shape[0], 2, 16, dtype=torch.int32, device=DEV)
    ws = qa.alloc_workspace(max(qa.paged_attn_workspace_bytes(2, 4, 2, 10 ** 5, 64), qa.paged_evict_workspace_bytes(2, 2, 64, 16), 256), DEV)
    none = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    dense = torch.randn(1, 4, 8, 64, dtype=torch.float16, device=DEV)
    for call in (
            lambda: qa.paged_append(x[:0], x[:0], G["k"], G["v"], G["table"], G["lens"], cu_seqlens=cu, workspace=ws),
            lambda: qa.paged_append(x[:0], x[:0], G["k"], G["v"], table, lens, workspace=ws),
            lambda: qa.paged_attn(none, G["k"], G["v"], table, lens, 10 ** 5, workspace=ws),
            lambda: qa.paged_evict(G["k"], G["v"], mass, pos, table, lens, 16, 64, workspace=ws),
            lambda: qa.scored_attn(dense[:, :, :0], dense, dense, workspace=ws)):
        ws.fill_(255)
        call()
        assert qa.read_device_status(ws) == 0


def test_append_leaves_out_what_has_no_place():
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([40, 40, 40], 2, 64, 16, torch.float16)      # three pages each: room for 48
    G = on_gpu(c)
    ws = qa.alloc_workspace(256, DEV)
    k = torch.ones(3, 2, 64, dtype=torch.float16, device=DEV)
    before = G["k"].clone()
    lens = torch.tensor([48, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    qa.paged_append(k, k, G["k"], G["v"], G["table"], lens, workspace=ws)
    assert qa.read_device_status(ws) == 12 and torch.equal(G["k"], before)
    table = G["table"].clone()
    table[:, 2] = torch.tensor([-1, c["k"].shape[0], 2 ** 31 - 1], dtype=torch.int32)
    qa.paged_append(k, k, G["k"], G["v"], table, G["lens"], workspace=ws)
    assert qa.read_device_status(ws) == 13 and torch.equal(G["k"], before)
    qa.paged_append(k, k, G["k"], G["v"], G["table"], G["lens"], workspace=ws)
    assert qa.read_device_status(ws) == 0 and not torch.equal(G["k"], before)


@pytest.mark.parametrize("lens", [[-3, 5, 7], [5, -10, 7], [5, 7, -2 ** 31], [-1, -2, -9]])
@pytest.mark.parametrize("told", [True, False])
def test_append_leaves_a_sequence_of_negative_length_alone(lens, told):
    # more new tokens than the length is below zero: the later ones must not land on what the sequence holds
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([20, 20, 20], 2, 64, 16, torch.float16, room=12)
    counts = [10, 11, 12]
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(sum(counts), 2, 64, generator=g).half() for _ in "kv")
    mass = torch.full((c["k"].shape[0], 2, 16), 5.0)
    kpos = torch.full((c["k"].shape[0], 2, 16), -3, dtype=torch.int32)
    cu = torch.tensor([0, 10, 21, 33], dtype=torch.int32)
    G, gm, gp = on_gpu(c), mass.to(DEV), kpos.to(DEV)
    ws = qa.alloc_workspace(256, DEV) if told else None
    qa.paged_append(k.to(DEV), v.to(DEV), G["k"], G["v"], G["table"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                    cu_seqlens=cu.to(DEV), mass=gm, key_positions=gp, workspace=ws)
    assert ws is None or qa.read_device_status(ws) == 12
    t = 0
    for b, n in enumerate(counts):
        for i in range(n if lens[b] >= 0 else 0):
            slot = lens[b] + i
            p, s = int(c["table"][b, slot // 16]), slot % 16
            c["k"][p, :, s], c["v"][p, :, s], mass[p, :, s], kpos[p, :, s] = k[t + i], v[t + i], 0.0, slot
        t += n
    assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])
    assert torch.equal(gm.cpu(), mass) and torch.equal(gp.cpu(), kpos)


EVICTIONS = [
    # lens, hkv, d, page, dtype, layout, budget, sink, recent, ties
    ([100, 64, 65, 3, 0], 2, 64, 16, torch.float16, "HND", 64, 4, 16, False),
    ([1500, 40], 3, 128, 7, torch.bfloat16, "NHD", 33, 0, 0, True),
    ([2, 9], 1, 20, 4, torch.bfloat16, "HND", 1, 0, 1, False),
    ([5000], 2, 72, 64, torch.float16, "NHD", 2500, 10, 1200, True),
    ([1030], 1, 64, 128, torch.float16, "HND", 1024, 0, 1024, False),
]


@pytest.mark.parametrize("lens,hkv,d,page,dtype,layout,budget,sink,recent,ties", EVICTIONS)
def test_evict(lens, hkv, d, page, dtype, layout, budget, sink, recent, ties):
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache(lens, hkv, d, page, dtype, layout, seed=9)
    g = torch.Generator().manual_seed(4)
    shape = (c["k"].shape[0], hkv, page)
    mass = torch.exp(3 * torch.randn(shape, generator=g))
    if ties:
        mass = torch.randint(0, 3, shape, generator=g).float()
        mass[torch.rand(shape, generator=g) < 0.1] = -0.0
        mass[torch.rand(shape, generator=g) < 0.05] = math.nan
        mass[torch.rand(shape, generator=g) < 0.05] = -math.inf
        mass[torch.rand(shape, generator=g) < 0.05] = math.inf
    pos = torch.zeros(shape, dtype=torch.int32)
    for b, n in enumerate(lens):
        p, s = ref.place(c, b, n)
        for h in range(hkv):
            pos[p, h, s] = torch.randperm(n, generator=g).to(torch.int32) + 100 * b
    G, gm, gp = on_gpu(c), mass.to(DEV), pos.to(DEV)
    ws = qa.alloc_workspace(qa.paged_evict_workspace_bytes(len(lens), hkv, max(lens), budget), DEV)
    ws.fill_(255)
    new = qa.paged_evict(G["k"], G["v"], gm, gp, G["table"], G["lens"], budget, max(lens), sink=sink, recent=recent,
                         tensor_layout=layout, workspace=ws)
    assert qa.read_device_status(ws) == 0
    want = ref.evict(c, mass, pos, budget, sink, recent)
    assert torch.equal(new.cpu(), want)
    assert torch.equal(gp.cpu(), pos)
    assert torch.equal(gm.cpu().view(torch.int32), mass.view(torch.int32))
    assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])


# (one CTA, two or four to a sequence, some of them without a slot; longer than the codes that shared memory holds;
# planes read four slots at a time and one at a time)
@pytest.mark.parametrize("lens,page,budget", [
    ([120001, 50000, 49152], 64, 30000), ([120001, 4097], 6, 1000), ([250001], 32, 400),
    ([60001, 50000] + [3] * 50, 64, 5000), ([60001, 49152] + [3] * 151, 16, 2000), ([60001] + [3] * 152, 10, 59000),
    ([5, 9, 4100, 4, 13], 4, 3)])
def test_evict_long_sequences(lens, page, budget):
    import quantized_attention_mean_gb300 as qa
    hkv, d = 1, 8
    c = ref.make_cache(lens, hkv, d, page, torch.float16, seed=3)
    g = torch.Generator().manual_seed(6)
    shape = (c["k"].shape[0], hkv, page)
    mass = torch.randint(0, 5000, shape, generator=g).float()    # ties across the chunks
    pos = torch.zeros(shape, dtype=torch.int32)
    for b, n in enumerate(lens):
        p, s = ref.place(c, b, n)
        pos[p, 0, s] = torch.arange(n, dtype=torch.int32)
    G, gm, gp = on_gpu(c), mass.to(DEV), pos.to(DEV)
    new = qa.paged_evict(G["k"], G["v"], gm, gp, G["table"], G["lens"], budget, max(lens), sink=min(4, budget - 1), recent=budget // 9)
    want = ref.evict(c, mass, pos, budget, min(4, budget - 1), budget // 9)
    assert torch.equal(new.cpu(), want) and torch.equal(gp.cpu(), pos) and torch.equal(gm.cpu(), mass)
    assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])


@pytest.mark.parametrize("bound", [4100, 18432, 18433, 60000])
@pytest.mark.parametrize("more", [0, 50, 160])
def test_evict_bounds_above_the_lengths(bound, more):
    # (the bound and the number of heads choose one CTA or a cluster to a sequence, most of it without a slot)
    import quantized_attention_mean_gb300 as qa
    hkv, d, page, budget = 1, 16, 8, 3
    lens = [5, 9, 4100, 4, 13, 0, 1] + [7] * more
    c = ref.make_cache(lens, hkv, d, page, torch.float16, seed=5)
    c["table"] = torch.cat([c["table"], torch.full((len(lens), bound // page), -9, dtype=torch.int32)], 1)
    g = torch.Generator().manual_seed(6)
    mass = torch.randint(0, 50, (c["k"].shape[0], hkv, page), generator=g).float()
    pos = torch.randint(0, 9999, mass.shape, generator=g, dtype=torch.int32)
    G, gm, gp = on_gpu(c), mass.to(DEV), pos.to(DEV)
    new = qa.paged_evict(G["k"], G["v"], gm, gp, G["table"], G["lens"], budget, bound, sink=1, recent=2)
    want = ref.evict(c, mass, pos, budget, 1, 2)
    assert torch.equal(new.cpu(), want) and torch.equal(gp.cpu(), pos) and torch.equal(gm.cpu(), mass)
    assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])


def test_evict_where_more_would_have_to_stay():
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([50], 1, 16, 8, torch.float16)
    shape = (c["k"].shape[0], 1, 8)
    mass, pos = torch.rand(shape, generator=torch.Generator().manual_seed(1)), torch.zeros(shape, dtype=torch.int32)
    G, gm, gp = on_gpu(c), mass.to(DEV), pos.to(DEV)             # every token at position 0
    new = qa.paged_evict(G["k"], G["v"], gm, gp, G["table"], G["lens"], 20, 50, sink=1)
    assert new.tolist() == [20] and torch.equal(G["k"].cpu(), c["k"]) and torch.equal(gm.cpu(), mass)


def test_evict_reports_bad_lengths_and_pages():
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([60, 60], 2, 64, 16, torch.float16)
    G = on_gpu(c)
    shape = (c["k"].shape[0], 2, 16)
    ws = qa.alloc_workspace(qa.paged_evict_workspace_bytes(2, 2, 60, 20), DEV)
    for what in ("length", "page"):
        mass, pos = torch.rand(shape, device=DEV), torch.zeros(shape, dtype=torch.int32, device=DEV)
        lens, table, k = G["lens"].clone(), G["table"].clone(), G["k"].clone()
        if what == "length":
            lens[0] = 65
        else:
            table[0, 3] = c["k"].shape[0]
        qa.paged_evict(k, G["v"].clone(), mass, pos, table, lens, 20, 60, workspace=ws)
        assert qa.read_device_status(ws) == (12 if what == "length" else 13)
        used = G["table"][0, :3].long()
        assert torch.equal(k[used], G["k"][used])                 # the bad sequence is left as it was


def test_evict_leaves_the_length_of_a_bad_sequence():
    import quantized_attention_mean_gb300 as qa
    c = ref.make_cache([60, 60, 60], 2, 64, 16, torch.float16)
    G = on_gpu(c)
    shape = (c["k"].shape[0], 2, 16)
    mass, pos = torch.rand(shape, device=DEV), torch.zeros(shape, dtype=torch.int32, device=DEV)
    lens, table = G["lens"].clone(), G["table"].clone()
    lens[0], table[1, 3] = 65, -1
    assert qa.paged_evict(G["k"], G["v"], mass, pos, table, lens, 20, 60).tolist() == [65, 60, 20]


def test_serving_loop_with_eviction():
    """Prompt, decode steps and evictions as a server runs them, against the same on the CPU."""
    import quantized_attention_mean_gb300 as qa
    B, hq, hkv, d, page, budget = 2, 4, 2, 64, 8, 24
    dtype = torch.float16
    g = torch.Generator().manual_seed(11)
    c = ref.make_cache([0, 0], hkv, d, page, dtype, room=64)
    c["k"].zero_(), c["v"].zero_()
    shape = (c["k"].shape[0], hkv, page)
    mass, pos = torch.zeros(shape), torch.zeros(shape, dtype=torch.int32)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625])
    G, gm, gp, gs = on_gpu(c), mass.to(DEV), pos.to(DEV), slopes.to(DEV)
    lens, told = G["lens"], torch.zeros(B, dtype=torch.int32)   # told: the next position of each sequence
    for step, counts in enumerate([[30, 11]] + [[1, 1]] * 12):
        T = sum(counts)
        k, v = (torch.randn(T, hkv, d, generator=g).to(dtype) for _ in "kv")
        q = torch.randn(B, hq, d, generator=g).to(dtype)
        cu = torch.tensor([0, counts[0], T], dtype=torch.int32)
        new_pos = torch.cat([told[b] + torch.arange(n) for b, n in enumerate(counts)]).to(torch.int32)
        qa.paged_append(k.to(DEV), v.to(DEV), G["k"], G["v"], G["table"], lens, cu_seqlens=cu.to(DEV), mass=gm,
                        key_positions=gp, positions=new_pos.to(DEV))
        lens = lens + torch.tensor(counts, dtype=torch.int32, device=DEV)
        told += torch.tensor(counts, dtype=torch.int32)
        out = qa.paged_attn(q.to(DEV), G["k"], G["v"], G["table"], lens, 64, slopes=gs, key_positions=gp,
                            q_positions=(told - 1).to(DEV), mass=gm)
        # the CPU's copy, from the device's state before the eviction
        c.update(k=G["k"].cpu(), v=G["v"].cpu(), lens=lens.cpu())
        r = decode_reference(c, q, 1 / math.sqrt(d), 0.0, slopes, gp.cpu(), told - 1, hkv)
        assert_close(out, r["out"], r["out_tol"], f"out of step {step}")
        mass, pos = gm.cpu(), gp.cpu()
        want = ref.evict(c, mass, pos, budget, 2, 6)
        lens = qa.paged_evict(G["k"], G["v"], gm, gp, G["table"], lens, budget, 64, sink=2, recent=6)
        assert torch.equal(lens.cpu(), want) and torch.equal(gp.cpu(), pos) and torch.equal(gm.cpu(), mass)
        assert torch.equal(G["k"].cpu(), c["k"]) and torch.equal(G["v"].cpu(), c["v"])


def test_evict_from_a_cache_without_pages():
    import quantized_attention_mean_gb300 as qa
    k = torch.empty(0, 2, 16, 64, dtype=torch.float16, device=DEV)
    mass, pos = torch.empty(0, 2, 16, device=DEV), torch.empty(0, 2, 16, dtype=torch.int32, device=DEV)
    ws = qa.alloc_workspace(qa.paged_evict_workspace_bytes(2, 2, 100, 10), DEV)
    for width in (0, 4):
        table, lens = torch.zeros(2, width, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
        assert qa.paged_evict(k, k, mass, pos, table, lens, 10, 100, workspace=ws).tolist() == [0, 0]
        assert qa.read_device_status(ws) == 0
    # tokens that no page holds: left as they were
    lens = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    assert qa.paged_evict(k, k, mass, pos, table, lens, 10, 100, workspace=ws).tolist() == [0, 40]
    assert qa.read_device_status(ws) == 13


def documented_loop(where):
    """The serving loop of the package's documentation, as code."""
    import quantized_attention_mean_gb300 as qa
    if where == "paged":
        text = qa.paged.__doc__
        text = text[text.index("    paged_append("):text.index("The cache is the caller's")]
    else:
        text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
        text = text[text.index("# prompts with capped"):]
        text = text[:text.index("```")]
    return textwrap.dedent(text)


@pytest.mark.parametrize("where", ["paged", "README"])
def test_the_documented_serving_loop_keeps_its_tokens(where):
    """Prompts, then steps of append, attention and eviction, as the documentation writes them: every step sees the tokens
    that were kept, at their own positions, with the newest; each head keeps its first, its last and `budget` in all."""
    import quantized_attention_mean_gb300 as qa
    B, hq, hkv, d, page, budget, longest, dtype = 2, 4, 2, 64, 16, 140, 150, torch.bfloat16
    prompt, steps = [150, 101], 60
    g = torch.Generator().manual_seed(21)
    rows = {n: torch.randn(B, longest + steps, hkv, d, generator=g).to(dtype) for n in "kv"}     # by position
    qs = torch.randn(B, longest + steps, hq, d, generator=g).to(dtype)
    slopes = torch.tensor([0.05, 0.02, 0.01, 0.0])
    c = ref.make_cache([0] * B, hkv, d, page, dtype, room=longest + 2)
    cache = on_gpu(c)
    new = lambda t, n: torch.stack([t[b, prompt[b] + n] for b in range(B)]).to(DEV)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    plane = (c["k"].shape[0], hkv, page)
    names = dict(q=qs[:, :longest].to(DEV), k=rows["k"][:, :longest].to(DEV), v=rows["v"][:, :longest].to(DEV),
                 held=(torch.arange(longest) < torch.tensor(prompt)[:, None]).to(DEV), k_cache=cache["k"],
                 v_cache=cache["v"], page_table=cache["table"], seq_lens=cache["lens"],
                 cu_seqlens=ints([0, prompt[0], sum(prompt)]), prompt_lens=ints(prompt), slopes=slopes.to(DEV),
                 mass=torch.full(plane, 3.0, device=DEV), positions=torch.full(plane, -5, dtype=torch.int32, device=DEV),
                 max_len=longest + 2, budget=budget,
                 steps=[(new(qs, n), new(rows["k"], n), new(rows["v"], n)) for n in range(steps)])
    if where == "paged":
        names.update(k=names["k"][names["held"]], v=names["v"][names["held"]])
    at = -1                                                                      # of the step
    kept = {(b, h): list(range(prompt[b])) for b in range(B) for h in range(hkv)}  # positions, by sequence and head

    def attn(*args, **kw):
        nonlocal at
        at += 1
        got = qa.paged_attn(*args, **kw)
        for (b, h), pos in kept.items():
            pos.append(prompt[b] + at)
            group = slice(h * hq // hkv, (h + 1) * hq // hkv)
            bias = -slopes[group, None].double() * (prompt[b] + at - torch.tensor(pos)).double()
            r = attend(qs[b, prompt[b] + at, group], rows["k"][b, pos, h], rows["v"][b, pos, h], d ** -0.5, 50.0, bias, dtype=dtype)
            assert_close(got[b, group], r["out"], r["out_tol"], f"sequence {b}, head {h}, step {at}")
        return got

    def evict(k_cache, v_cache, mass, positions, table, lens, *args, **kw):
        new_lens = qa.paged_evict(k_cache, v_cache, mass, positions, table, lens, *args, **kw)
        for (b, h), pos in kept.items():
            n = min(len(pos), budget)
            assert int(new_lens[b]) == n
            p, s = ref.place(c, b, n)
            left = positions.cpu()[p, h, s].tolist()
            assert len(set(left)) == n and set(left) <= set(pos)
            assert set(range(4)) | set(range(max(0, prompt[b] + at - 127), prompt[b] + at + 1)) <= set(left)
            kept[b, h] = left
        return new_lens

    calls = dict(paged_append=qa.paged_append, paged_attn=attn, paged_evict=evict, scored_attn=qa.scored_attn)
    exec(documented_loop(where), {**names, **calls, "qa": types.SimpleNamespace(**calls)})
    assert at == steps - 1 and all(len(p) == budget for p in kept.values())


def test_decode_step_in_a_graph_and_on_another_stream():
    import quantized_attention_mean_gb300 as qa
    lens = [500, 33, 64]
    c = ref.make_cache(lens, 2, 128, 16, torch.bfloat16, room=4)
    G = on_gpu(c)
    q = torch.randn(3, 8, 128).bfloat16().to(DEV)
    k = torch.randn(3, 2, 128).bfloat16().to(DEV)
    ws = qa.alloc_workspace(qa.paged_attn_workspace_bytes(3, 8, 2, 600, 128), DEV)
    out = torch.empty_like(q)
    lens_new = G["lens"] + 1

    def step(stream=None):
        qa.paged_append(k, k, G["k"], G["v"], G["table"], G["lens"], stream=stream)
        qa.paged_attn(q, G["k"], G["v"], G["table"], lens_new, 600, out=out, workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, eager)
    # outputs that the call allocates on another stream belong to that stream
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
    mine = qa.paged_attn(q, G["k"], G["v"], G["table"], lens_new, 600, stream=side)
    side.synchronize()
    assert torch.equal(mine, out)
