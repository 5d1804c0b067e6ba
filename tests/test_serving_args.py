"""What the calls for serving from an 8-bit cache refuse, on the CPU: the binding's checks and the C ABI's statuses
(both come before any device work)."""

import ctypes

import pytest
import torch

import quantized_attention_mean_gb300 as qa

S8, E4 = torch.int8, torch.float8_e4m3fn


# ---- norms and rotation
def test_rope_checks():
    q, k = torch.zeros(5, 4, 64, dtype=torch.float16), torch.zeros(5, 2, 64, dtype=torch.float16)
    f = torch.ones(32)

    def refuses(kind, match, *a, **kw):
        with pytest.raises(kind, match=match):
            qa.qk_norm_rope(*(a or (q, k)), **kw)
    refuses(ValueError, "CUDA device")
    refuses(ValueError, "4-D", q[0], k[0])
    refuses(ValueError, "packed rows", tensor_layout="HND")
    refuses(ValueError, "tensor_layout", tensor_layout="DNH")
    refuses(TypeError, "dtype", q, k.bfloat16())
    refuses(TypeError, "dtype", q.float(), k.float())
    refuses(ValueError, "tokens and head_dim", q, k[:4])
    refuses(ValueError, "tokens and head_dim", q, k[..., :32])
    refuses(ValueError, "at most head_dim", inv_freq=torch.ones(33))
    refuses(ValueError, "inv_freq must", inv_freq=f.double())
    refuses(ValueError, "positions must", positions=torch.zeros(4, dtype=torch.int32))
    refuses(ValueError, "positions must", positions=torch.zeros(5))
    refuses(ValueError, "positions must", positions=torch.zeros(1, 5, dtype=torch.int32))
    refuses(ValueError, "q_weight must", q_weight=torch.ones(63))
    refuses(ValueError, "k_weight must", k_weight=torch.ones(64, dtype=torch.bfloat16))
    refuses(TypeError, "share one dtype", q_weight=torch.ones(64), k_weight=torch.ones(64, dtype=torch.float16))
    for eps in (-1.0, float("inf"), float("nan")):
        refuses(ValueError, "eps", eps=eps)
    refuses(ValueError, "q_out must have", q_out=q[:4])
    refuses(ValueError, "k_out must have", k_out=k.bfloat16())
    q4 = torch.zeros(2, 5, 4, 64, dtype=torch.float16)
    refuses(ValueError, "positions must", q4, q4, positions=torch.zeros(5, 2, dtype=torch.int32))
    refuses(ValueError, "tokens and head_dim", q4, q4[:1])
    with pytest.raises(ValueError, match="last dimension"):
        from quantized_attention_mean_gb300 import rope
        rope._view(q.transpose(0, 2), True, False)


def test_rope_outputs_that_overlap():
    x = torch.zeros(6, 8, 64, dtype=torch.float16)
    q, k = x[:, :4], x[:, 4:6]

    def call(match, **kw):
        with pytest.raises(ValueError, match=match):
            qa.qk_norm_rope(q, k, **kw)
    call("CUDA device", q_out=q, k_out=k)                              # each in its own place
    call("CUDA device", q_out=torch.zeros_like(q), k_out=x[:, 6:])
    call("q_out must be its input", q_out=x[:, 1:5])
    call("k_out must be its input", k_out=q[:, :2])
    call("k_out must be its input", k_out=x[:, 5:7])
    out = torch.zeros(6, 6, 64, dtype=torch.float16)
    call("CUDA device", q_out=out[:, :4], k_out=out[:, 4:])
    call("must not overlap", q_out=out[:, :4], k_out=out[:, 3:5])
    h = torch.zeros(2, 6, 8, 64, dtype=torch.float16).transpose(1, 2)  # HND views of NHD rows
    with pytest.raises(ValueError, match="CUDA device"):
        qa.qk_norm_rope(h[:, :4], h[:, 4:6], tensor_layout="HND", q_out=h[:, :4], k_out=h[:, 4:6])
    with pytest.raises(ValueError, match="its input"):
        qa.qk_norm_rope(h[:, :4], h[:, 4:6], tensor_layout="HND", q_out=h[:, 4:8])


# ---- page tables
def test_page_table_checks():
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    table = torch.zeros(2, 4, dtype=torch.int32)

    def assign(**kw):
        a = dict(page_table=table, seq_lens=i(0, 0), add_lens=i(1, 1), free_pages=i(1, 2, 3), free_count=i(3), page_size=4, max_tokens=2)
        a.update(kw)
        return qa.paged_assign(**a)

    def release(**kw):
        a = dict(page_table=table, seq_lens=i(0, 0), keep_lens=i(0, 0), free_pages=i(1, 2, 3), free_count=i(3), page_size=4)
        a.update(kw)
        return qa.paged_release(**a)
    for call in (assign, release):
        for kw, match in ((dict(page_table=table.long()), "page_table"), (dict(page_table=table[0]), "page_table"),
                          (dict(page_table=table.T), "page_table"), (dict(seq_lens=i(0)), "seq_lens"),
                          (dict(seq_lens=torch.zeros(2)), "seq_lens"), (dict(free_pages=torch.zeros(3)), "free_pages"),
                          (dict(free_count=i(1, 2)), "free_count"), (dict(page_size=0), "page_size"),
                          (dict(page_size=2 ** 31), "page_size"), (dict(), "CUDA device"),
                          (dict(workspace=torch.zeros(256)), "workspace")):
            with pytest.raises(ValueError, match=match):
                call(**kw)
    for kw, match in ((dict(add_lens=i(1)), "add_lens"), (dict(max_tokens=-1), "max_tokens"), (dict(max_tokens=2 ** 31), "max_tokens"),
                      (dict(next_positions=i(1)), "next_positions")):
        with pytest.raises(ValueError, match=match):
            assign(**kw)
    with pytest.raises(ValueError, match="keep_lens"):
        release(keep_lens=i(1, 2, 3))


# ---- the 8-bit cache
def cache(pages=6, hkv=2, size=16, d=64, kt=S8, vt=E4, batch=3, width=2, blocks=2):
    return dict(k_cache=torch.zeros(pages, hkv, size, d, dtype=torch.uint8).view(kt),
                v_cache=torch.zeros(pages, hkv, size, d, dtype=torch.uint8).view(vt), k_scales=torch.zeros(pages, hkv, blocks),
                v_scales=torch.zeros(pages, hkv, blocks), page_table=torch.zeros(batch, width, dtype=torch.int32),
                seq_lens=torch.zeros(batch, dtype=torch.int32))


def test_cache_checks():
    q, k = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(3, 2, 64, dtype=torch.float16)
    cu = torch.zeros(4, dtype=torch.int32)
    calls = [lambda **kw: qa.paged_attn_q8(q, max_seq_len=32, **{**cache(), **kw}),
             lambda **kw: qa.paged_append_q8(k, k, **{**cache(), **kw}),
             lambda **kw: qa.paged_read_q8(cu_seqlens=cu, tokens=3, **{**cache(), **kw})]
    z = torch.zeros
    for call in calls:
        for kw, kind, match in (
                (dict(v_cache=z(5, 2, 16, 64, dtype=S8)), ValueError, "one shape"),
                (dict(k_cache=z(6, 2, 16, 64, dtype=torch.float16)), TypeError, "int8 or"),
                (dict(v_cache=z(6, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e5m2)), TypeError, "int8 or"),
                (dict(seq_lens=z(3, dtype=torch.int64)), TypeError, "int32"),
                (dict(page_table=z(2, 3, dtype=torch.int32).T), ValueError, "page_table must"),
                (dict(seq_lens=z(2, dtype=torch.int32)), ValueError, "seq_lens must"),
                (dict(tensor_layout="DHN"), ValueError, "tensor_layout"),
                (dict(k_scales=z(6, 2, 3)), ValueError, "divides page_size"),
                (dict(k_scales=z(6, 2, 0)), ValueError, "divides page_size"),
                (dict(k_scales=z(6, 2)), ValueError, "divides page_size"),
                (dict(k_scales=z(6, 3, 2)), ValueError, "k_scales must"),
                (dict(v_scales=z(6, 2, 4)), ValueError, "v_scales must"),
                (dict(v_scales=z(6, 2, 2, dtype=torch.float64)), ValueError, "v_scales must"),
                (dict(k_cache=z(6, 2, 16, 128, dtype=S8)[..., ::2]), ValueError, "last dimension"),
                (dict(), ValueError, "CUDA device")):
            with pytest.raises(kind, match=match):
                call(**kw)


def test_attn_append_and_read_checks():
    c = cache()
    q, k = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(5, 2, 64, dtype=torch.float16)
    cu = torch.zeros(4, dtype=torch.int32)
    for a, kw, kind, match in (
            (q[:2], {}, ValueError, "q must be"), (q[..., :32], {}, ValueError, "q must be"), (q.float(), {}, TypeError, "float16"),
            (q, dict(out=q[..., :32]), ValueError, "out must"), (q, dict(max_seq_len=-1), ValueError, "CUDA|max_seq_len"),
            (q, dict(slopes=torch.zeros(5)), ValueError, "slopes must"), (q, dict(q_positions=torch.zeros(3)), ValueError, "q_positions"),
            (q, dict(return_lse=True, lse=torch.zeros(4, 3)), ValueError, "lse must")):
        with pytest.raises(kind, match=match):
            qa.paged_attn_q8(a, **{**dict(max_seq_len=32), **c, **kw})
    for a, kw, kind, match in (((k, k), {}, ValueError, "one token"), ((k, k[:4]), {}, ValueError, "k and v must"),
                               ((k.bfloat16(), k), {}, TypeError, "one dtype"), ((k.float(), k.float()), {}, TypeError, "float16"),
                               ((k[:, :1], k[:, :1]), {}, ValueError, "k and v must"),
                               ((k, k), dict(cu_seqlens=cu[:3]), ValueError, "cu_seqlens")):
        with pytest.raises(kind, match=match):
            qa.paged_append_q8(*a, **c, **kw)
    for kw, kind, match in ((dict(tokens=-1), ValueError, "tokens"), (dict(dtype=torch.float32), TypeError, "dtype"),
                            (dict(cu_seqlens=cu.long()), ValueError, "cu_seqlens"), (dict(starts=cu), ValueError, "starts"),
                            (dict(k_out=k), ValueError, "k_out"), (dict(v_out=k.bfloat16()[:3]), ValueError, "CUDA device")):
        with pytest.raises(kind, match=match):
            qa.paged_read_q8(**{**dict(cu_seqlens=cu, tokens=3), **c, **kw})


# ---- the C ABI: fake addresses are never dereferenced, validation stops before any launch
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from quantized_attention_mean_gb300 import _lib, build
    build.build()
    return _lib.load()


def c_cache(**over):
    from quantized_attention_mean_gb300._lib import SageQ8Cache
    a = dict(k=FAKE, ks=(2 * 16 * 64, 16 * 64, 64), v=FAKE, vs=(2 * 16 * 64, 16 * 64, 64), sk=FAKE, sv=FAKE, kt=0, vt=1, pages=6,
             size=16, block=8, table=FAKE, ts=2, width=2, lens=FAKE)
    a.update(over)
    return SageQ8Cache(a["k"], *a["ks"], a["v"], *a["vs"], a["sk"], a["sv"], a["kt"], a["vt"], a["pages"], a["size"], a["block"],
                       a["table"], a["ts"], a["width"], a["lens"])


def test_c_cache_statuses(lib):
    from quantized_attention_mean_gb300._lib import SagePacked
    t = SagePacked(FAKE, 256, 64)

    def attn(c=None, q=t, o=t, batch=3, hq=4, hkv=2, maxn=32, d=64, dtype=0, layout=0, cap=0.0, ws=FAKE * 16, wsb=1 << 40):
        c = c or c_cache()
        return lib.sage_paged_attn_q8(ctypes.byref(q), ctypes.byref(c), ctypes.byref(o), None, None, None, batch, hq, hkv, maxn, d,
                                      dtype, layout, 0.0, cap, ctypes.c_void_p(ws), wsb, None)

    def append(c=None, k=t, cu=FAKE, batch=3, tokens=5, d=64, dtype=0, layout=0, ws=0, wsb=0, **kw):
        c = c or c_cache()
        return lib.sage_paged_append_q8(ctypes.byref(k), ctypes.byref(t), ctypes.byref(c), ctypes.c_void_p(cu), batch, tokens, 2, d,
                                        dtype, layout, ctypes.c_void_p(ws), wsb, None)

    def read(c=None, k=t, cu=FAKE, starts=0, batch=3, tokens=5, d=64, dtype=0, layout=0, ws=0, wsb=0):
        c = c or c_cache()
        return lib.sage_paged_read_q8(ctypes.byref(k), ctypes.byref(t), ctypes.byref(c), ctypes.c_void_p(cu), ctypes.c_void_p(starts),
                                      batch, tokens, 2, d, dtype, layout, ctypes.c_void_p(ws), wsb, None)
    for call in (attn, append, read):
        assert call(d=129) == 2 and call(d=0) == 2
        assert call(dtype=2) == 3
        assert call(layout=2) == 1
        assert call(c_cache(kt=2)) == 3 and call(c_cache(vt=-1)) == 3
        assert call(c_cache(block=0)) == 1 and call(c_cache(block=5)) == 1 and call(c_cache(block=32)) == 1
        assert call(c_cache(size=0)) == 1 and call(c_cache(table=0)) == 1 and call(c_cache(lens=FAKE + 2)) == 1
        assert call(c_cache(sk=0)) == 1 and call(c_cache(sv=FAKE + 2)) == 1 and call(c_cache(k=0)) == 1
        assert call(c_cache(vs=(1, -1, 1))) == 4
        assert call(c_cache(size=65536, width=65536, block=1)) == 1    # slots past 32 bits
    assert attn(hq=3) == 5 and attn(maxn=-1) == 1 and attn(cap=-1.0) == 1 and attn(batch=0) == 0
    assert attn(hkv=0) == 1
    assert attn(q=SagePacked(0, 1, 1)) == 1 and attn(q=SagePacked(FAKE + 1, 256, 64)) == 4
    assert attn(o=SagePacked(FAKE, 0, 64)) == 4 and attn(o=SagePacked(FAKE, 256, 0)) == 4
    assert attn(ws=FAKE * 16 + 8) == 6 and attn(ws=FAKE * 16, wsb=128) == 6
    assert attn(ws=0, maxn=10 ** 6) == 6                               # the line's pieces need a workspace
    assert append(cu=0) == 1 and append(tokens=-1) == 1 and append(tokens=0) == 0 and append(batch=0, cu=FAKE) == 0
    assert append(ws=FAKE * 16, wsb=128) == 6 and append(ws=FAKE * 16 + 4, wsb=1024) == 6
    assert append(k=SagePacked(FAKE + 1, 128, 64)) == 4 and append(k=SagePacked(FAKE, -128, 64)) == 4 and append(k=SagePacked(0, 1, 1)) == 1
    assert read(cu=0) == 1 and read(starts=FAKE + 1) == 1 and read(tokens=0) == 0 and read(tokens=-1) == 1
    assert read(k=SagePacked(FAKE, 0, 64)) == 4 and read(k=SagePacked(FAKE, 128, 0)) == 4


def test_c_rope_statuses(lib):
    from quantized_attention_mean_gb300._lib import SageView
    t = SageView(FAKE, 4096, 256, 64)

    def rope(q=t, o=t, freq=FAKE, w=0, wt=0, batch=2, hq=4, hkv=2, n=16, d=64, rot=64, dtype=0, layout=1, eps=1e-6, pos=0, ps=0):
        return lib.sage_qk_norm_rope(ctypes.byref(q), ctypes.byref(t), ctypes.byref(o), ctypes.byref(t), ctypes.c_void_p(pos), ps,
                                     ctypes.c_void_p(freq), ctypes.c_void_p(w), None, wt, batch, hq, hkv, n, d, rot, dtype, layout, 0,
                                     eps, None)
    assert rope(d=0) == 2 and rope(d=130) == 2
    assert rope(dtype=2) == 3 and rope(w=FAKE, wt=1) == 3
    assert rope(layout=2) == 1 and rope(rot=63) == 1 and rope(rot=66) == 1 and rope(rot=-2) == 1 and rope(freq=0) == 1
    assert rope(eps=-1.0) == 1 and rope(eps=float("nan")) == 1 and rope(eps=float("inf")) == 1 and rope(ps=-1) == 1
    assert rope(hq=0) == 1 and rope(hkv=0) == 1 and rope(n=-1) == 1
    assert rope(n=0) == 0 and rope(batch=0) == 0
    assert rope(q=SageView(0, 1, 1, 1)) == 1 and rope(q=SageView(FAKE + 1, 4096, 256, 64)) == 4
    assert rope(q=SageView(FAKE, -1, 256, 64)) == 4 and rope(o=SageView(FAKE, 4096, 0, 64)) == 4
    assert rope(pos=FAKE + 2) == 1 and rope(freq=FAKE + 1) == 1 and rope(w=FAKE + 2, wt=2) == 1


def test_c_page_table_statuses(lib):
    p = ctypes.c_void_p
    F = FAKE

    def assign(table=F, stride=4, width=4, lens=F * 2, add=F * 3, nxt=0, free=F * 4, count=F * 5, pages=8, size=16, batch=2, most=4,
               new=F * 6, held=F * 7, cu=F * 8, pos=F * 9, slots=F * 10, out=F * 11, ws=0, wsb=0):
        return lib.sage_paged_assign(p(table), stride, width, p(lens), p(add), p(nxt), p(free), p(count), pages, size, batch, most, p(new),
                                     p(held), p(cu), p(pos), p(slots), p(out), p(ws), wsb, None)

    def release(table=F, stride=4, width=4, lens=F * 2, add=F * 3, free=F * 4, count=F * 5, pages=8, size=16, batch=2, out=F * 11,
                ws=F * 16, wsb=1 << 20):
        return lib.sage_paged_release(p(table), stride, width, p(lens), p(add), p(free), p(count), pages, size, batch, p(out), p(ws), wsb,
                                      None)
    for call in (assign, release):
        assert call(size=0) == 1 and call(batch=-1) == 1 and call(batch=65536) == 1 and call(pages=-1) == 1 and call(width=-1) == 1
        assert call(lens=0) == 1 and call(add=F + 2) == 1 and call(free=0) == 1 and call(count=0) == 1 and call(out=F * 5) == 1
        assert call(table=0) == 1 and call(stride=3) == 4 and call(size=1 << 30) == 1
        assert call(ws=F * 16 + 4, wsb=1 << 20) == 6 and call(ws=F * 16, wsb=64) == 6
    assert assign(most=-1) == 1 and assign(new=0) == 1 and assign(held=F * 7 + 1) == 1 and assign(cu=0) == 1
    assert assign(pos=0) == 1 and assign(slots=F + 4) == 1 and assign(nxt=F + 1) == 1
    assert assign(new=F * 2) == 1 and assign(held=F * 3 - 4) == 1      # results over the lengths they come from
    assert release(ws=0) == 6 and release(wsb=256) == 6
    assert lib.sage_paged_release_workspace_size(2) == 512 and lib.sage_paged_release_workspace_size(-1) == 0
    assert lib.sage_paged_release_workspace_size(0) == 256
