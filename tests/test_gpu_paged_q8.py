"""An 8-bit paged cache: append and read against plain loops, attention against float64 over the same codes."""

import math

import pytest
import torch

import paged_reference as ref
import q8_reference as q8
from attn_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
S8, E4 = torch.int8, torch.float8_e4m3fn


def on_gpu(c):
    return {n: (t.to(DEV) if torch.is_tensor(t) else t) for n, t in c.items()}


def planes(G):
    return G["k"], G["v"], G["ks"], G["vs"]


def same(x, y):
    return torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8).cpu())


# ------------------------------------------------------------------------------------- attention
CASES = [
    # lens, hq, hkv, d, page, block, dtype, codes of k and v, layout, cap, slopes
    ([1], 1, 1, 64, 16, 16, torch.float16, S8, E4, "HND", 0.0, False),
    ([1, 0, 17, 64, 65], 8, 2, 128, 16, 4, torch.bfloat16, S8, E4, "HND", 0.0, False),
    ([300, 5, 0, 129], 14, 2, 128, 7, 7, torch.bfloat16, E4, S8, "NHD", 30.0, False),       # group of 7, pages of 7
    ([63, 2000, 1], 16, 1, 64, 48, 16, torch.float16, E4, E4, "NHD", 0.0, True),
    ([500, 777], 40, 2, 80, 32, 32, torch.float16, S8, S8, "HND", 20.0, True),              # group of 20: two row blocks
    ([130, 1, 90], 6, 3, 33, 8, 8, torch.bfloat16, S8, E4, "HND", 0.0, False),              # rows of single bytes
    ([130, 33], 4, 2, 36, 8, 2, torch.bfloat16, E4, S8, "HND", 0.0, False),                 # rows of 4 bytes
    ([513, 90], 9, 1, 72, 24, 1, torch.float16, S8, E4, "NHD", 0.0, False),                 # rows of 8 bytes
    ([4097] * 3, 32, 8, 128, 64, 64, torch.bfloat16, S8, E4, "HND", 0.0, False),
    ([20001], 8, 8, 96, 128, 32, torch.bfloat16, E4, E4, "NHD", 50.0, True),                # one sequence over many CTAs
    ([3] * 150, 4, 4, 64, 4, 4, torch.float16, S8, S8, "HND", 0.0, False),
    ([0, 0], 4, 2, 64, 16, 16, torch.float16, S8, E4, "HND", 0.0, False),
    ([100, 257], 12, 1, 16, 64, 16, torch.float16, E4, S8, "HND", 0.0, True),
    ([300, 0, 1000, 77], 8, 4, 64, 32, 16, torch.bfloat16, S8, E4, "NHD", 0.0, True),       # four heads side by side
    ([5, 700], 48, 4, 64, 16, 16, torch.float16, E4, S8, "NHD", 0.0, False),                # and twelve queries each
    ([129, 640, 31], 36, 2, 128, 16, 8, torch.bfloat16, S8, E4, "NHD", 25.0, False),        # two row blocks, two heads side by side
    ([1000] * 9, 24, 2, 128, 32, 32, torch.float16, E4, E4, "HND", 0.0, False),             # twelve queries, head_dim 128
    ([2, 64, 65, 128], 6, 6, 48, 24, 8, torch.bfloat16, S8, S8, "NHD", 0.0, True),
    ([1, 31, 32, 33, 100, 600, 0, 95] * 5, 16, 4, 128, 16, 16, torch.bfloat16, S8, E4, "HND", 0.0, False),  # short ones: four heads
    ([63, 64, 65, 500] * 6, 6, 6, 64, 16, 16, torch.float16, E4, S8, "HND", 0.0, True),                     # and two to an item
    ([900, 33, 0, 1200, 64], 32, 8, 96, 16, 8, torch.bfloat16, E4, S8, "NHD", 20.0, True),   # four, by six units of channels
    ([700, 1, 40, 129] * 9, 8, 4, 120, 24, 24, torch.float16, S8, E4, "NHD", 0.0, False),
    ([2000, 64, 31] * 13, 4, 4, 32, 32, 32, torch.bfloat16, S8, S8, "HND", 0.0, True),       # two units
    ([2000, 64, 31] * 13, 40, 4, 36, 16, 4, torch.float16, E4, E4, "NHD", 0.0, False),
    ([2000, 64, 31] * 13, 40, 4, 72, 16, 4, torch.bfloat16, S8, E4, "HND", 0.0, False),
    ([500, 77], 12, 1, 20, 8, 8, torch.bfloat16, S8, E4, "HND", 0.0, True),
    ([500, 77], 20, 2, 90, 8, 8, torch.float16, E4, S8, "NHD", 0.0, False),
]


# (a bound far above the lengths takes the form for long sequences)
@pytest.mark.parametrize("bound", [0, 10 ** 5])
@pytest.mark.parametrize("lens,hq,hkv,d,page,block,dtype,kt,vt,layout,cap,biased", CASES)
def test_decode(lens, hq, hkv, d, page, block, dtype, kt, vt, layout, cap, biased, bound):
    import quantized_attention_mean_gb300 as qa
    bound = max(max(lens), bound)
    c = q8.make_cache(lens, hkv, d, page, block, kt, vt, layout, seed=len(lens) + d, spread=1.0)
    q = (torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(5)) * 2).to(dtype)
    slopes = 2.0 ** (-torch.arange(1, hq + 1).float() / 4) if biased else None
    G = on_gpu(c)
    ws = qa.alloc_workspace(qa.paged_attn_q8_workspace_bytes(len(lens), hq, hkv, bound, d), DEV)
    ws.fill_(255)
    out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, tensor_layout=layout, softcap=cap,
                                slopes=None if slopes is None else slopes.to(DEV), return_lse=True, workspace=ws)
    assert qa.read_device_status(ws) == 0
    r = q8.attend(c, q, 1 / math.sqrt(d), cap, slopes, hkv=hkv)
    assert_close(out, r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("bound", [700, 10 ** 5])
@pytest.mark.parametrize("d,kt,vt", [(64, S8, E4), (128, E4, S8)])
def test_scales_of_very_different_blocks(d, kt, vt, bound):
    # V's scales over 2^+-30 and some of them 0: a weight and its scale together decide what a key adds
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache([700, 81], 2, d, 16, 4, kt, vt, seed=3, spread=1.0)
    g = torch.Generator().manual_seed(9)
    c["vs"] = torch.exp2(torch.randint(-30, 31, c["vs"].shape, generator=g).float())
    c["vs"][torch.rand(c["vs"].shape, generator=g) < 0.1] = 0.0
    c["ks"][torch.rand(c["ks"].shape, generator=g) < 0.1] = 0.0
    q = (torch.randn(2, 6, d, generator=g) * 40).bfloat16()              # bf16: the largest result is about 2^38
    G = on_gpu(c)
    out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, return_lse=True)
    r = q8.attend(c, q, d ** -0.5, hkv=2)
    assert_close(out, r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")
    c["vs"].zero_()
    out, lse = qa.paged_attn_q8(q.to(DEV), G["k"], G["v"], G["ks"], c["vs"].to(DEV), G["table"], G["lens"], bound, return_lse=True)
    assert (out == 0).all()
    assert_close(lse, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("lens,bound", [([700, 81], 700), ([700, 81], 10 ** 5), ([20001, 3], 20001)])
@pytest.mark.parametrize("d,hq,vt", [(64, 6, E4), (128, 24, S8)])
def test_values_near_the_largest(d, hq, vt, lens, bound):
    # values of 2^127, as 16-bit ones may be: their sums pass fp32, their averages do not
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache(lens, 2, d, 16, 16, S8, vt, seed=d)
    c["v"] = q8.to_codes(torch.randint(100, 128, c["v"].shape, generator=torch.Generator().manual_seed(d)).float(), vt)
    c["vs"].fill_(2.0 ** 120)
    q = torch.randn(2, hq, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    G = on_gpu(c)
    out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, return_lse=True)
    r = q8.attend(c, q, d ** -0.5, hkv=2)
    assert_close(out, r["out"], r["out_tol"], "out")
@pytest.mark.parametrize("bound", [700, 10 ** 5])
@pytest.mark.parametrize("lo,hi,gap", [(-110, 20, 122), (-10, 120, 122), (-60, 60, 124), (-60, 100, 140), (-110, 110, 200)])
@pytest.mark.parametrize("d,hq,kt,vt", [(64, 6, S8, E4), (128, 24, E4, S8)])
def test_v_scales_that_outweigh_the_scores(d, hq, kt, vt, lo, hi, gap, bound):
    # keys with the top score and V scales of 2^lo beside keys 2^gap less likely with V scales of 2^hi, which make the result
    import quantized_attention_mean_gb300 as qa
    hkv, lens = 2, [700, 81]
    c = q8.make_cache(lens, hkv, d, 16, 4, kt, vt, seed=lo + d)
    g = torch.Generator().manual_seed(gap)
    k = torch.randint(-3, 4, c["k"].shape, generator=g).float()
    k[..., 0] = 0
    c["ks"].fill_(gap * math.log(2) * d ** 0.5 / (96 * 64))             # 96 of channel 0, where q is 64: `gap` in base 2
    c["vs"].fill_(2.0 ** hi)
    for b, n in enumerate(lens):
        for t in range(5, n, 64):
            p, s = int(c["table"][b, t // 16]), t % 16
            k[p, :, s, 0] = 96
            c["vs"][p, :, s // 4] = 2.0 ** lo
    c["k"] = q8.to_codes(k, kt)
    q = torch.randn(2, hq, d, generator=g) * 4
    q[..., 0] = 64
    q = q.bfloat16()
    G = on_gpu(c)
    out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, return_lse=True)
    lift = max(0, gap - hi)                                             # the bound's absolute part lies below what is compared
    r = q8.attend(dict(c, vs=(c["vs"].double() * 2.0 ** lift)), q, d ** -0.5, hkv=hkv)
    assert_close(out.double() * 2.0 ** lift, r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("bound", [2000, 10 ** 5])
@pytest.mark.parametrize("d,hq,vt", [(64, 8, E4), (64, 16, S8), (128, 8, S8), (128, 16, E4)])
def test_a_sink_with_a_small_scale_before_a_long_tail(d, hq, vt, bound):
    # one key of 32 draws nearly all attention and adds nothing; V scales beside it are 2^8 of its own, at keys of no weight; the
    # others, 2^-18 to 2^-22 of its weight and all alike, make the result: their weights keep their bits beside the sink's
    import quantized_attention_mean_gb300 as qa
    lens = [2000, 320]
    c = q8.make_cache(lens, 1, d, 16, 1, S8, vt, seed=d + hq)
    k = torch.zeros(c["k"].shape)
    v = torch.randint(1, 100, c["v"].shape, generator=torch.Generator().manual_seed(d)).float()
    c["ks"].fill_(20 * math.log(2) * d ** 0.5 / (100 * 64))             # 100 of channel 0, where q is 64: 20 in base 2
    c["vs"].fill_(2.0 ** 4)
    for b, n in enumerate(lens):
        for t in range(0, n, 8):
            p, s = int(c["table"][b, t // 16]), t % 16
            if t % 32 == 0:
                k[p, :, s, 0] = 100
                v[p, :, s] = 0
            else:
                k[p, :, s, 0] = -127
                c["vs"][p, :, s] = 2.0 ** 12
    c["k"], c["v"] = q8.to_codes(k, S8), q8.to_codes(v, vt)
    q = torch.zeros(2, hq, d)
    q[..., 0] = 58 + torch.arange(hq) * (14 / hq)
    q = q.half()
    G = on_gpu(c)
    out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, return_lse=True)
    r = q8.attend(c, q, d ** -0.5)
    assert_close(out, r["out"], r["out_tol"], "out")
    assert_close(lse, r["lse"], r["lse_tol"], "lse")


def test_queries_of_every_size():
    # rows of q far above and below fp16's range, and of channels of very different sizes
    import quantized_attention_mean_gb300 as qa
    d = 64
    c = q8.make_cache([90], 1, d, 16, 16, S8, S8, seed=4)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(1, 7, d, generator=g)
    q[0, 1] *= 1e6
    q[0, 2] *= 1e-30
    q[0, 3] = 0
    q[0, 4, 1:] *= 1e-9
    q[0, 5] *= 2.0 ** -126
    q = q.bfloat16()
    q[0, 6] = torch.finfo(torch.bfloat16).tiny / 4
    c["ks"] *= 1e-6
    G = on_gpu(c)
    for scale in (d ** -0.5, 1e-3):
        out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], 90, sm_scale=scale, return_lse=True)
        r = q8.attend(c, q, scale)
        assert_close(out, r["out"], r["out_tol"], "out")
        assert_close(lse, r["lse"], r["lse_tol"], "lse")


def test_slices_strides_positions_and_scale():
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache([200, 33], 2, 64, 16, 8, S8, S8, seed=2)
    hkv, d, hq = 2, 64, 8
    g = torch.Generator().manual_seed(1)
    qpos = torch.tensor([5001, 77], dtype=torch.int32)
    q = torch.randn(2, hq, d, generator=g).half()
    slopes = torch.linspace(0.001, 0.02, hq)
    G = on_gpu(c)
    for gap in (16, 8, 4, 1):                                        # loads of as many bytes
        wide = torch.zeros(c["k"].shape[0], hkv, 16, 2 * d + 2 * gap, dtype=torch.int8, device=DEV)
        kc, vc = wide[..., gap:gap + d], wide[..., 2 * gap + d:]
        kc.copy_(G["k"])
        vc.copy_(G["v"])
        qw = torch.zeros(2, 2 * hq, d + 1, dtype=torch.float16, device=DEV)
        qw[:, ::2, 1:] = q.to(DEV)
        ow = torch.full((2, 2 * hq, d + 1), 9.0, dtype=torch.float16, device=DEV)
        lse = torch.empty(2, hq, device=DEV)
        for bound in (999, 10 ** 5):
            qa.paged_attn_q8(qw[:, ::2, 1:], kc, vc, G["ks"], G["vs"], G["table"], G["lens"], bound, sm_scale=0.3,
                             slopes=slopes.to(DEV), q_positions=qpos.to(DEV), return_lse=True, out=ow[:, ::2, 1:], lse=lse)
            r = q8.attend(c, q, 0.3, 0.0, slopes, qpos, hkv)
            assert_close(ow[:, ::2, 1:], r["out"], r["out_tol"], "out")
            assert_close(lse, r["lse"], r["lse_tol"], "lse")
            assert (ow[:, 1::2] == 9).all() and (ow[..., 0] == 9).all()


@pytest.mark.parametrize("bound", [70, 10 ** 5])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 64), (72, 16)])
def test_garbage_behind_the_end(d, page, bound):
    # slots and scales behind a sequence's end and unused pages hold NaN: nothing of them may show
    import quantized_attention_mean_gb300 as qa
    lens = [70, 5]
    c = q8.make_cache(lens, 2, d, page, 1, E4, E4, seed=6)
    used = torch.zeros(c["k"].shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        p, s = ref.place(c, b, n)
        used[p, s] = True
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    r = q8.attend(c, q, 1 / math.sqrt(d), hkv=2)
    for w in "kv":
        c[w].view(torch.uint8)[(~used)[:, None, :].expand(-1, 2, -1)] = 0x7f
        c[w + "s"][(~used)[:, None, :].expand(-1, 2, -1)] = math.nan
    G = on_gpu(c)
    out = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound)
    assert_close(out, r["out"], r["out_tol"], "out")


@pytest.mark.parametrize("bound", [96, 10 ** 5])
def test_bad_lengths_and_pages_are_told(bound):
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache([40, 40, 40, 40], 2, 64, 16, 16, S8, E4, seed=8)
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(3)).half()
    ws = qa.alloc_workspace(qa.paged_attn_q8_workspace_bytes(4, 4, 2, bound, 64), DEV)
    r = q8.attend(c, q, 0.125, hkv=2)
    G = on_gpu(c)
    for bad in (-1, 49, 2 ** 31 - 1):
        lens = G["lens"].clone()
        lens[1] = bad
        out, lse = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], lens, bound, return_lse=True, workspace=ws)
        assert qa.read_device_status(ws) == 12
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        for b in (0, 2, 3):
            assert_close(out[b], r["out"][b], r["out_tol"][b], "out")
    for bad in (-1, c["k"].shape[0]):
        table = G["table"].clone()
        table[2, 1] = bad
        out = qa.paged_attn_q8(q.to(DEV), *planes(G), table, G["lens"], bound, workspace=ws)
        assert qa.read_device_status(ws) == 13
        z = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in c.items()}
        at = int(z["table"][2, 1])
        z["k"][at], z["ks"][at], z["vs"][at] = 0, 0.0, 0.0             # rows of zeros
        w = q8.attend(z, q, 0.125, hkv=2)
        assert_close(out, w["out"], w["out_tol"], "out")
    qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], G["lens"], bound, workspace=ws)
    assert qa.read_device_status(ws) == 0


def test_the_same_bits_every_time():
    # ranges that end anywhere, joined by another kernel: results do not depend on which part is done first
    import quantized_attention_mean_gb300 as qa
    for layout, d in (("HND", 128), ("NHD", 64)):
        c = q8.make_cache([5000, 1, 333, 9001], 4, d, 16, 16, S8, E4, layout, seed=5)
        G = on_gpu(c)
        q = torch.randn(4, 20, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
        for bound in (9001, 10 ** 6):
            first = qa.paged_attn_q8(q, *planes(G), G["table"], G["lens"], bound, tensor_layout=layout, return_lse=True)
            for _ in range(20):
                again = qa.paged_attn_q8(q, *planes(G), G["table"], G["lens"], bound, tensor_layout=layout, return_lse=True)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_streams_at_once():
    # calls whose workspaces come from the allocator run side by side
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache([4000, 2500], 8, 128, 32, 32, S8, E4, seed=9)
    G = on_gpu(c)
    qs = [torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(i)).bfloat16().to(DEV) for i in range(2)]
    want = [qa.paged_attn_q8(q, *planes(G), G["table"], G["lens"], 10 ** 5) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(30):
        for i, st in enumerate(streams):
            got[i].append(qa.paged_attn_q8(qs[i], *planes(G), G["table"], G["lens"], 10 ** 5, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_empty_cache_and_result_over_the_query():
    import quantized_attention_mean_gb300 as qa
    k = torch.empty(0, 2, 16, 64, dtype=S8, device=DEV)
    s = torch.empty(0, 2, 1, device=DEV)
    table, lens = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    q = torch.randn(2, 4, 64, dtype=torch.float16, device=DEV)
    for bound in (0, 10 ** 5):
        out, lse = qa.paged_attn_q8(q, k, k, s, s, table, lens, bound, return_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    c = q8.make_cache([300, 40], 2, 64, 16, 16, S8, E4)
    G = on_gpu(c)
    for bound in (300, 10 ** 5):
        want = qa.paged_attn_q8(q, *planes(G), G["table"], G["lens"], bound)
        both = q.clone()
        qa.paged_attn_q8(both, *planes(G), G["table"], G["lens"], bound, out=both)
        assert torch.equal(both, want)


# ------------------------------------------------------------------------------------- append, read
APPENDS = [
    # held, new, hkv, d, page, block, dtype, codes of k and v, layout
    ([0], [1], 1, 64, 16, 16, torch.float16, S8, E4, "HND"),
    ([5, 16, 0, 31], [1, 1, 1, 1], 2, 128, 16, 16, torch.bfloat16, S8, E4, "HND"),
    ([0, 3, 0, 17], [40, 0, 1, 70], 3, 128, 32, 8, torch.bfloat16, E4, S8, "NHD"),
    ([7, 1], [9, 200], 2, 72, 64, 64, torch.float16, S8, E4, "NHD"),
    ([7, 1], [9, 30], 2, 33, 7, 7, torch.float16, E4, S8, "HND"),      # rows of single bytes
    ([2, 0], [3, 20], 1, 36, 6, 3, torch.bfloat16, S8, S8, "HND"),
    ([4, 250], [300, 30], 1, 64, 256, 256, torch.float16, E4, E4, "HND"),  # more rows than stay in registers
    ([0, 9], [5, 6], 2, 16, 4, 1, torch.bfloat16, S8, E4, "NHD"),      # a scale per token
    ([1] * 40, [2] * 40, 5, 128, 8, 4, torch.bfloat16, S8, E4, "HND"),
    ([0, 0], [0, 0], 2, 64, 16, 16, torch.float16, S8, E4, "HND"),
    ([3, 0, 20], [64, 31, 100], 2, 120, 64, 32, torch.bfloat16, S8, E4, "NHD"),     # a block by two warps
    ([5, 100, 0], [400, 27, 128], 3, 128, 128, 128, torch.float16, E4, S8, "HND"),  # by eight
    ([129], [390], 1, 96, 192, 192, torch.bfloat16, S8, S8, "NHD"),
    ([6, 0, 63], [60, 2, 70], 3, 36, 64, 64, torch.float16, S8, E4, "NHD"),         # runs of four channels
    ([6, 0, 63], [60, 2, 70], 2, 20, 64, 8, torch.bfloat16, E4, S8, "HND"),
    ([1, 0, 15, 40], [70, 33, 1, 1], 4, 32, 32, 1, torch.bfloat16, S8, S8, "HND"),  # rows of four lanes
    ([1, 0, 15, 40], [70, 33, 1, 1], 2, 24, 48, 16, torch.float16, E4, S8, "NHD"),
    ([30, 2], [80, 200], 2, 32, 64, 64, torch.bfloat16, S8, E4, "HND"),
    ([30, 2], [80, 200], 2, 12, 40, 40, torch.float16, S8, S8, "NHD"),
    ([2, 0, 9], [17, 40, 1], 2, 64, 12, 6, torch.bfloat16, S8, E4, "HND"),          # two blocks of six to a window
]


@pytest.mark.parametrize("held,new,hkv,d,page,block,dtype,kt,vt,layout", APPENDS)
def test_append_and_read(held, new, hkv, d, page, block, dtype, kt, vt, layout):
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(d + page)
    c = q8.make_cache(held, hkv, d, page, block, kt, vt, layout, seed=d, room=max(new) + 1)
    T = sum(new)
    # growing magnitudes, so that blocks are joined by larger tokens, and by smaller ones
    k, v = ((torch.randn(T + 2, hkv, d, generator=g) * torch.exp(1.5 * torch.randn(T + 2, hkv, 1, generator=g))).to(dtype) for _ in "kv")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    G = on_gpu(c)
    ws = qa.alloc_workspace(256, DEV).fill_(255)
    step = all(n == 1 for n in new)
    rows = T if step else T + 2                                        # rows behind the last sequence are left out
    qa.paged_append_q8(k[:rows].to(DEV), v[:rows].to(DEV), *planes(G), G["table"], G["lens"],
                       cu_seqlens=None if step else torch.tensor(cu, dtype=torch.int32, device=DEV), tensor_layout=layout, workspace=ws)
    assert qa.read_device_status(ws) == 0
    q8.append(c, k, v, cu)
    for w in "kv":
        assert same(G[w], c[w]), f"codes of {w}"
        assert torch.equal(G[w + "s"].cpu(), c[w + "s"]), f"scales of {w}"
    # all tokens out again, from the first and from some later slot on
    for starts in (None, [min(n, 3) for n in held]):
        lens = [n + m for n, m in zip(held, new)]
        count = [n - s for n, s in zip(lens, starts or [0] * len(lens))]
        out = [0]
        for n in count:
            out.append(out[-1] + n)
        got = qa.paged_read_q8(*planes(G), G["table"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                               torch.tensor(out, dtype=torch.int32, device=DEV), out[-1] + 2,
                               starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV),
                               dtype=dtype, tensor_layout=layout, workspace=ws)
        assert qa.read_device_status(ws) == 0
        for w, y in zip("kv", got):
            want = torch.zeros(out[-1] + 2, hkv, d, dtype=dtype)
            for b, n in enumerate(lens):
                for h in range(hkv):
                    x = q8.values(c, w, b, h, n, (starts or [0] * len(lens))[b])
                    want[out[b]:out[b + 1], h] = x.float().to(dtype)   # code * scale is rounded to 32 bits, then to 16
            assert torch.equal(y.cpu(), want), w


def test_appending_one_by_one_or_all_at_once():
    # E4M3 codes agree but for subnormals; int8 codes are off by half a step for each time the scale grew
    import quantized_attention_mean_gb300 as qa
    n, hkv, d, page = 48, 2, 64, 16
    g = torch.Generator().manual_seed(11)
    x = torch.randn(n, hkv, d, generator=g).half()
    x = torch.where(x.abs() < 0.05, torch.tensor(0.05).half(), x)       # no value is subnormal as a code
    for dt in (E4, S8):
        caches = []
        for steps in ([n], [1] * n, [5, 20, 1, 22]):
            c = q8.make_cache([0], hkv, d, page, page, dt, dt, seed=1, room=n)
            G = on_gpu(c)
            at = 0
            for m in steps:
                lens = torch.tensor([at], dtype=torch.int32, device=DEV)
                rows = x[at:at + m].to(DEV)
                qa.paged_append_q8(rows, rows, *planes(G), G["table"], lens, cu_seqlens=torch.tensor([0, m], dtype=torch.int32, device=DEV))
                at += m
            caches.append(G)
            lens = torch.tensor([n], dtype=torch.int32, device=DEV)
            cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            k, _ = qa.paged_read_q8(*planes(G), G["table"], lens, cu, n, dtype=torch.float16)
            p, s = ref.place(c, 0, n)
            scale = G["ks"].cpu()[p, :, 0].double()
            off = (k.cpu().double() - x.double()).abs()
            if dt == E4:
                assert (off <= x.double().abs() * (2.0 ** -4 + 2.0 ** -11)).all()
            else:
                growths = 16 if len(steps) == n else len(steps)
                assert (off <= (scale * (0.5 + 0.5 * growths))[..., None] * 1.001 + x.double().abs() * 2.0 ** -11).all()
        p, s = (t[:n] for t in ref.place(c, 0, n))
        for other in caches[1:]:
            assert torch.equal(other["ks"].cpu()[p, :, 0], caches[0]["ks"].cpu()[p, :, 0])
            if dt == E4:
                a, b = (t["k"].view(torch.uint8).cpu()[p, :, s] for t in (caches[0], other))
                assert torch.equal(a, b)


def test_what_has_no_place_is_left_out():
    import quantized_attention_mean_gb300 as qa
    hkv, d, page = 2, 64, 8
    c = q8.make_cache([3, 3, 3, 3], hkv, d, page, 8, S8, E4, seed=5, room=8)
    before = {n: t.clone() if torch.is_tensor(t) else t for n, t in c.items()}
    k = torch.randn(20, hkv, d, generator=torch.Generator().manual_seed(1)).half()
    G = on_gpu(c)
    width = c["table"].shape[1]
    lens = torch.tensor([-1, width * page - 2, 3, 3], dtype=torch.int32, device=DEV)
    table = G["table"].clone()
    table[2, 0] = c["k"].shape[0]
    table[1, -1] = -1
    ws = qa.alloc_workspace(256, DEV)
    cu = torch.tensor([0, 4, 8, 12, 14], dtype=torch.int32, device=DEV)
    qa.paged_append_q8(k.to(DEV), k.to(DEV), *planes(G), table, lens, cu_seqlens=cu, workspace=ws)
    assert qa.read_device_status(ws) in (12, 13)
    want = {n: t.clone() if torch.is_tensor(t) else t for n, t in before.items()}
    want["lens"] = torch.tensor([0, 0, 0, 3], dtype=torch.int32)        # the last sequence alone has a place for its two
    q8.append(want, k[12:14], k[12:14], [0, 0, 0, 0, 2])
    for w in "kv":
        assert same(G[w], want[w]) and torch.equal(G[w + "s"].cpu(), want[w + "s"])
    # reads: behind the length, of a bad page, of a negative first slot
    lens = torch.tensor([3, 3, 3, 5], dtype=torch.int32, device=DEV)
    starts = torch.tensor([1, -1, 0, 4], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 4, 6, 8, 9], dtype=torch.int32, device=DEV)
    out = torch.full((11, hkv, 2 * d), 7.0, dtype=torch.float16, device=DEV)
    qa.paged_read_q8(*planes(G), table, lens, cu, 11, starts=starts, dtype=torch.float16, k_out=out[..., :d], v_out=out[..., d:],
                     workspace=ws)
    assert qa.read_device_status(ws) in (12, 13)
    for w, y in zip("kv", (out[..., :d], out[..., d:])):
        x = torch.zeros(11, hkv, d, dtype=torch.float16)
        for h in range(hkv):
            x[0:2, h] = q8.values(want, w, 0, h, 3, 1).half()
            x[8:9, h] = q8.values(want, w, 3, h, 5, 4).half()
        # (row 4 is slot -1; row 5 is slot 0 of the second, whose table's first page is sound)
        for h in range(hkv):
            x[5, h] = q8.values(want, w, 1, h, 1, 0).half()[0]
        assert torch.equal(y.cpu(), x)


@pytest.mark.parametrize("lead", [1, 3, 20, 200])
@pytest.mark.parametrize("hkv,d,page,block,kt,vt", [(2, 64, 16, 16, S8, E4), (1, 128, 128, 128, E4, S8), (2, 32, 32, 1, S8, S8),
                                                    (3, 72, 64, 64, S8, E4)])
def test_rows_before_the_first_sequence_are_left_out(hkv, d, page, block, kt, vt, lead):
    # cu_seqlens of a slice of a batch: the rows of the sequences before it are not written, all others are; the status says so
    import quantized_attention_mean_gb300 as qa
    held, new = [5, 16, 0], [40, 3, 70]
    c = q8.make_cache(held, hkv, d, page, block, kt, vt, seed=lead, room=max(new) + 1)
    cu = [lead, lead + 40, lead + 43, lead + 113]
    k, v = (torch.randn(cu[-1] + 2, hkv, d, generator=torch.Generator().manual_seed(i)).bfloat16() for i in range(2))
    G = on_gpu(c)
    ws = qa.alloc_workspace(256, DEV).fill_(255)
    qa.paged_append_q8(k.to(DEV), v.to(DEV), *planes(G), G["table"], G["lens"],
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), workspace=ws)
    assert qa.read_device_status(ws) == 12
    q8.append(c, k, v, cu)
    for w in "kv":
        assert same(G[w], c[w]), f"codes of {w}"
        assert torch.equal(G[w + "s"].cpu(), c[w + "s"]), f"scales of {w}"


def test_broadcast_keys_and_zero_tokens_and_tiny_values():
    import quantized_attention_mean_gb300 as qa
    hkv, d = 4, 64
    for dt in (S8, E4):
        c = q8.make_cache([0, 0], hkv, d, 16, 16, dt, dt, seed=3, room=16)
        c["ks"].fill_(9.0)                                              # what a page's last owner left
        G = on_gpu(c)
        k = torch.zeros(6, 1, d, dtype=torch.bfloat16)
        k[3:] = torch.randn(3, 1, d, generator=torch.Generator().manual_seed(1)).bfloat16() * 2.0 ** -104
        v = torch.zeros(6, hkv, d, dtype=torch.bfloat16)
        v[1] = 3e38
        cu = [0, 3, 6]
        qa.paged_append_q8(k.to(DEV).expand(6, hkv, d), v.to(DEV), *planes(G), G["table"], G["lens"],
                           cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        q8.append(c, k.expand(6, hkv, d), v, cu)
        for w in "kv":
            assert same(G[w], c[w]) and torch.equal(G[w + "s"].cpu(), c[w + "s"])


def test_a_cache_past_32_bits():
    # pages whose rows lie more than 2^32 bytes into the cache
    import quantized_attention_mean_gb300 as qa
    pages, hkv, page, d = 300000, 1, 128, 128                           # 4.9 GB each
    k = torch.empty(pages, hkv, page, d, dtype=S8, device=DEV)
    v = torch.empty(pages, hkv, page, d, dtype=E4, device=DEV)
    ks, vs = (torch.empty(pages, hkv, 8, device=DEV) for _ in "kv")
    at = torch.tensor([299999, 1, 299998, 270000], dtype=torch.int32)
    c = q8.make_cache([400], hkv, d, page, 16, S8, E4)
    c["table"][0] = torch.arange(4, dtype=torch.int32)
    c["lens"][0] = 0
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(400, hkv, d, generator=g).half() for _ in "kv"]
    q8.append(c, *new, [0, 400])
    c["lens"][0] = 400
    table, lens = at[None].to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 400], dtype=torch.int32, device=DEV)
    qa.paged_append_q8(*(t.to(DEV) for t in new), k, v, ks, vs, table, lens, cu_seqlens=cu)
    held = at.long().to(DEV)
    p, s = ref.place(c, 0, 400)
    assert same(k.view(torch.uint8)[held][p, :, s], c["k"].view(torch.uint8)[p, :, s])
    q = torch.randn(1, 4, d, generator=g).half()
    for bound in (400, 10 ** 5):
        out = qa.paged_attn_q8(q.to(DEV), k, v, ks, vs, table, lens + 400, bound)
        r = q8.attend(c, q, d ** -0.5, hkv=hkv)
        assert_close(out, r["out"], r["out_tol"], "out")
    a, b = qa.paged_read_q8(k, v, ks, vs, table, lens + 400, cu, 400, dtype=torch.float16)
    assert torch.equal(a[:, 0].cpu(), q8.values(c, "k", 0, 0, 400).float().half())
    assert torch.equal(b[:, 0].cpu(), q8.values(c, "v", 0, 0, 400).float().half())


def test_calls_with_nothing_to_do_say_so():
    # a workspace that held another call's error: an empty call leaves no status of it
    import quantized_attention_mean_gb300 as qa
    c = q8.make_cache([30, 5], 2, 64, 16, 16, S8, E4)
    G = on_gpu(c)
    none = {n: (t[:0] if n in ("table", "lens") else t) for n, t in G.items()}
    x = torch.randn(2, 2, 64, dtype=torch.float16, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    ws = qa.alloc_workspace(qa.paged_attn_q8_workspace_bytes(2, 4, 2, 10 ** 5, 64), DEV)
    calls = [
        lambda **kw: qa.paged_append_q8(x[:0], x[:0], *planes(G), G["table"], G["lens"], cu_seqlens=cu, workspace=ws, **kw),
        lambda **kw: qa.paged_append_q8(x[:0], x[:0], *planes(none), none["table"], none["lens"], workspace=ws, **kw),
        lambda **kw: qa.paged_append_q8(x, x, *planes(none), none["table"], none["lens"], cu_seqlens=cu[:1], workspace=ws, **kw),
        lambda **kw: qa.paged_read_q8(*planes(G), G["table"], G["lens"], cu, 0, workspace=ws, **kw),
        lambda **kw: qa.paged_attn_q8(torch.empty(0, 4, 64, dtype=torch.float16, device=DEV), *planes(none), none["table"],
                                      none["lens"], 10 ** 5, workspace=ws, **kw),
    ]
    side = torch.cuda.Stream()
    for call in calls:
        ws.fill_(255)
        call()
        assert qa.read_device_status(ws) == 0
        ws.fill_(255)
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        assert qa.read_device_status(ws, side) == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        ws.fill_(255)
        graph.replay()
        assert qa.read_device_status(ws) == 0
        call_ws = qa.alloc_workspace(512, DEV)[64:]
        with pytest.raises((qa.SageError, ValueError)):
            qa.paged_read_q8(*planes(G), G["table"], G["lens"], cu, 0, workspace=call_ws)
    assert same(G["k"], c["k"]) and torch.equal(G["ks"].cpu(), c["ks"])


@pytest.mark.parametrize("bound", [300, 10 ** 5])
@pytest.mark.parametrize("kt,vt,block,offset", [(S8, E4, 16, 0.0), (S8, S8, 64, 2.0), (E4, E4, 16, 0.5), (S8, E4, 1, 4.0)])
def test_against_attention_over_the_unrounded_keys_and_values(kt, vt, block, offset, bound):
    # what eight bits cost: scores move by half a step of every channel of a key, values by half a step of their own
    import quantized_attention_mean_gb300 as qa
    lens, hq, hkv, d, page = [300, 77], 8, 2, 64, 64
    c = q8.make_cache([0, 0], hkv, d, page, block, kt, vt, seed=1, room=300)
    g = torch.Generator().manual_seed(block)
    k = (torch.randn(377, hkv, d, generator=g) + offset * torch.randn(hkv, d, generator=g)).half()
    v = torch.randn(377, hkv, d, generator=g).half()
    q = torch.randn(2, hq, d, generator=g).half()
    G = on_gpu(c)
    cu = [0, 300, 377]
    qa.paged_append_q8(k.to(DEV), v.to(DEV), *planes(G), G["table"], G["lens"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    out = qa.paged_attn_q8(q.to(DEV), *planes(G), G["table"], torch.tensor(lens, dtype=torch.int32, device=DEV), bound)
    c.update(k=G["k"].cpu(), v=G["v"].cpu(), ks=G["ks"].cpu(), vs=G["vs"].cpu(), lens=torch.tensor(lens, dtype=torch.int32))
    kernel = q8.attend(c, q, d ** -0.5, hkv=hkv)["out_tol"]

    def half_step(x, scale, dt):
        # an int8 code is off by half a scale (and the reciprocal's rounding), an E4M3 one by 2^-4 of itself or half of 2^-9
        return (scale * 0.5001).expand_as(x) if dt == S8 else torch.maximum(x.abs() * 2.0 ** -4, scale * 2.0 ** -10)

    for b, n in enumerate(lens):
        p, s = ref.place(c, b, n)
        for h in range(hkv):
            x, kk, vv = (t.double() for t in (q[b, h * 4:h * 4 + 4], k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h]))
            dk, dv = (half_step(t, c[w + "s"][p, h, s // block].double()[:, None], dt) for t, w, dt in ((kk, "k", kt), (vv, "v", vt)))
            weights = torch.softmax(x @ kk.T * d ** -0.5, -1)
            moved = (x.abs() @ dk.T * d ** -0.5).amax(-1, keepdim=True)
            tol = torch.expm1(2 * moved) * (weights @ vv.abs()) + torch.exp(2 * moved) * (weights @ dv)
            assert_close(out[b, h * 4:h * 4 + 4], weights @ vv, tol + kernel[b, h * 4:h * 4 + 4], "out")


# ------------------------------------------------------------------------------------- together
def freqs(n):
    return (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float().to(DEV)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_a_serving_loop(layout):
    """Prompts in chunks, then tokens one by one: pages from the stack, norms and rotation, the append, attention of the
    chunks over what the cache gives back, attention of the tokens over the cache, pages back at the end."""
    import quantized_attention_mean_gb300 as qa
    B, hq, hkv, d, page, block, pages = 3, 8, 2, 64, 16, 16, 40
    g = torch.Generator().manual_seed(12)
    shape = (pages, hkv, page, d) if layout == "HND" else (pages, page, hkv, d)
    kc, vc = torch.zeros(shape, dtype=S8, device=DEV), torch.zeros(shape, dtype=E4, device=DEV)
    ks, vs = (torch.zeros(pages, hkv, page // block, device=DEV) for _ in "kv")
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    free, count = torch.arange(pages, dtype=torch.int32, device=DEV), torch.tensor([pages], dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    wq, wk, freq = (1 + 0.1 * torch.randn(d, generator=g)).half().to(DEV), torch.ones(d, dtype=torch.float16, device=DEV), freqs(32)
    kept = [torch.zeros(0, hkv, 2, d, dtype=torch.float16) for _ in range(B)]  # rotated keys and values of each sequence
    chunks = [[70, 33, 1], [20, 50, 40]] + [[1, 1, 1]] * 6
    for i, new in enumerate(chunks):
        T = sum(new)
        x = torch.randn(T, hq + 2 * hkv, d, generator=g).half().to(DEV)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        a = qa.paged_assign(table, lens, torch.tensor(new, dtype=torch.int32, device=DEV), free, count, page, T)
        qa.qk_norm_rope(q, k, a.positions, freq, wq, wk, q_out=q, k_out=k)
        qa.paged_append_q8(k, v, kc, vc, ks, vs, table, a.held_lens, None if i > 1 else a.cu_seqlens, tensor_layout=layout)
        before, lens, count = lens, a.seq_lens, a.free_count
        cu = a.cu_seqlens.tolist()
        for b in range(B):
            kept[b] = torch.cat((kept[b], torch.stack((k, v), 2)[cu[b]:cu[b + 1]].cpu()))
        assert lens.tolist() == [t.shape[0] for t in kept]
        c = dict(k=kc.cpu(), v=vc.cpu(), ks=ks.cpu(), vs=vs.cpu(), table=table.cpu(), lens=lens.cpu(), layout=layout, size=page,
                 block=block)
        # the slot map: where the append has put each token
        for b in range(B):
            t = torch.arange(before[b], lens[b])
            p, s = c["table"][b, t // page].long(), t % page
            assert a.slots[cu[b]:cu[b + 1]].tolist() == (p * page + s).tolist()
        if i < 2:
            total = [0]
            for n in lens.tolist():
                total.append(total[-1] + n)
            rk, rv = qa.paged_read_q8(kc, vc, ks, vs, table, lens, torch.tensor(total, dtype=torch.int32, device=DEV), total[-1],
                                      dtype=torch.float16, tensor_layout=layout)
            for b in range(B):
                want, got = kept[b].double(), torch.stack((rk, rv), 2)[total[b]:total[b + 1]].cpu().double()
                # int8 of a block's largest, E4M3 of each value (its smallest ones to half of 2^-9 of their scale)
                assert (want[:, :, 0] - got[:, :, 0]).abs().max() <= 0.03 * want[:, :, 0].abs().max()
                assert ((want[:, :, 1] - got[:, :, 1]).abs() <= want[:, :, 1].abs() * 0.0635 + 2.0 ** -9 * c["vs"].max()).all()
                o = qa.scored_attn(q[None, cu[b]:cu[b + 1]], rk[None, total[b]:total[b + 1]], rv[None, total[b]:total[b + 1]],
                                   tensor_layout="NHD", is_causal=True, q_offset=int(before[b]))
                # the chunk's last row sees all: the decode call over the cache says the same
                last = qa.paged_attn_q8(q[cu[b + 1] - 1:cu[b + 1]], kc, vc, ks, vs, table[b:b + 1], lens[b:b + 1], 200,
                                        tensor_layout=layout)
                assert (o[0, -1:].double() - last.double()).abs().max() <= 0.01
        else:
            out, lse = qa.paged_attn_q8(q, kc, vc, ks, vs, table, lens, 200, tensor_layout=layout, return_lse=True)
            r = q8.attend(c, q.cpu(), d ** -0.5, hkv=hkv)
            assert_close(out, r["out"], r["out_tol"], "out")
            assert_close(lse, r["lse"], r["lse_tol"], "lse")
    held = sum(-(-t.shape[0] // page) for t in kept)
    assert count.item() == pages - held
    count = qa.paged_release(table, lens, torch.zeros_like(lens), free, count, page)
    assert count.item() == pages and sorted(free.tolist()) == list(range(pages))


@pytest.mark.parametrize("bound", [128, 10 ** 5])
def test_a_step_in_a_graph_and_on_another_stream(bound):
    import quantized_attention_mean_gb300 as qa
    B, hq, hkv, d, page = 3, 8, 2, 128, 16
    c = q8.make_cache([100, 31, 16], hkv, d, page, page, S8, E4, seed=7, room=20)
    need = c["table"].shape[1]
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().to(DEV)
    freq, one = freqs(64), torch.ones(B, dtype=torch.int32, device=DEV)
    free = torch.tensor([0], dtype=torch.int32, device=DEV)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = qa.alloc_workspace(qa.paged_attn_q8_workspace_bytes(B, hq, hkv, bound, d), DEV)

    def state():
        G = on_gpu(c)
        # pages of the room that make_cache gave are in the table already: the stack is the pages of the cache, empty
        return dict(G, free=torch.zeros(c["k"].shape[0], dtype=torch.int32, device=DEV), lens=G["lens"].clone())

    def step(s, x):
        a = qa.paged_assign(s["table"], s["lens"], one, s["free"], none, page, B)
        q, k = qa.qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], a.positions, freq)
        qa.paged_append_q8(k, x[:, hq + hkv:], *planes(s), s["table"], a.held_lens)
        out = qa.paged_attn_q8(q, *planes(s), s["table"], a.seq_lens, bound, workspace=ws)
        return out, a.seq_lens

    # the third sequence needs a page and finds none: its token is left out, the others are served
    eager = state()
    want, new_lens = step(eager, x)
    assert new_lens.tolist() == [101, 32, 16]
    s, first = state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, lens = step(s, x)
    for _ in range(2):
        for n in ("k", "v", "ks", "vs", "table"):
            s[n].copy_(first[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lens, new_lens)
        assert all(same(s[n], eager[n]) for n in ("k", "v", "ks", "vs"))
    side = torch.cuda.Stream()
    other = state()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, _ = step(other, x)
    side.synchronize()
    assert torch.equal(out, want)
    assert need >= 2 and free.numel() == 1
