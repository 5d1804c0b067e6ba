"""What the paged cache's calls refuse, on the CPU: the binding's checks and the C ABI's statuses
(both come before any device work)."""

import ctypes

import pytest
import torch

import quantized_attention_mean_gb300 as qa


def cache(pages=6, hkv=2, size=16, d=64, dtype=torch.float16, batch=3, width=2):
    k = torch.zeros(pages, hkv, size, d, dtype=dtype)
    return dict(k_cache=k, v_cache=k.clone(), page_table=torch.zeros(batch, width, dtype=torch.int32),
                seq_lens=torch.zeros(batch, dtype=torch.int32))


def planes(pages=6, hkv=2, size=16):
    return dict(mass=torch.zeros(pages, hkv, size), key_positions=torch.zeros(pages, hkv, size, dtype=torch.int32))


def test_cache_checks():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    call = lambda **kw: qa.paged_attn(q, max_seq_len=32, **{**cache(), **kw})  # noqa: E731
    with pytest.raises(ValueError, match="one shape"):
        call(v_cache=torch.zeros(5, 2, 16, 64, dtype=torch.float16))
    with pytest.raises(TypeError, match="share one dtype"):
        call(v_cache=torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="int32"):
        call(seq_lens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="page_table must"):
        call(page_table=torch.zeros(2, 3, dtype=torch.int32).T)
    with pytest.raises(ValueError, match="seq_lens must"):
        call(seq_lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="tensor_layout"):
        call(tensor_layout="DHN")
    with pytest.raises(ValueError, match="mass must"):
        call(mass=torch.zeros(6, 16, 2))
    with pytest.raises(ValueError, match="key_positions must"):
        call(key_positions=torch.zeros(6, 2, 16))
    with pytest.raises(ValueError, match="CUDA device"):
        call()


def test_attn_checks():
    c = cache()
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="q must be"):
        qa.paged_attn(torch.zeros(2, 4, 64, dtype=torch.float16), max_seq_len=32, **c)
    with pytest.raises(ValueError, match="q must be"):
        qa.paged_attn(torch.zeros(3, 4, 32, dtype=torch.float16), max_seq_len=32, **c)
    with pytest.raises(TypeError, match="dtype"):
        qa.paged_attn(q.bfloat16(), max_seq_len=32, **c)
    with pytest.raises(ValueError, match="out must"):
        qa.paged_attn(q, max_seq_len=32, out=torch.zeros(3, 4, 32, dtype=torch.float16), **c)
    for n in (-1, 2 ** 31):
        with pytest.raises(ValueError, match="CUDA|max_seq_len"):
            qa.paged_attn(q, max_seq_len=n, **c)
    with pytest.raises(ValueError, match="slopes must"):
        qa.paged_attn(q, max_seq_len=32, slopes=torch.zeros(5), **c)
    with pytest.raises(ValueError, match="q_positions must"):
        qa.paged_attn(q, max_seq_len=32, q_positions=torch.zeros(3), **c)
    with pytest.raises(ValueError, match="lse must"):
        qa.paged_attn(q, max_seq_len=32, return_lse=True, lse=torch.zeros(4, 3), **c)


def test_append_checks():
    c = cache()
    k = torch.zeros(5, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="one token"):
        qa.paged_append(k, k, **c)
    with pytest.raises(ValueError, match="k and v must be"):
        qa.paged_append(k, k[:4], **c)
    with pytest.raises(ValueError, match="k and v must be"):
        qa.paged_append(k[:, :1], k[:, :1], **c)
    with pytest.raises(TypeError, match="dtype"):
        qa.paged_append(k.bfloat16(), k.bfloat16(), **c)
    with pytest.raises(ValueError, match="cu_seqlens must"):
        qa.paged_append(k, k, cu_seqlens=torch.zeros(3, dtype=torch.int32), **c)
    with pytest.raises(ValueError, match="key_positions plane"):
        qa.paged_append(k, k, cu_seqlens=torch.zeros(4, dtype=torch.int32),
                        positions=torch.zeros(5, dtype=torch.int32), **c)
    with pytest.raises(ValueError, match="CUDA device"):
        qa.paged_append(k[:3], k[:3], **c)


def test_evict_checks():
    c, p = cache(), planes()
    for budget, sink, recent in ((0, 0, 0), (4, 3, 2), (4, -1, 0), (4, 0, -1)):
        with pytest.raises(ValueError, match="budget"):
            qa.paged_evict(budget=budget, sink=sink, recent=recent, max_seq_len=32, **c, **p)
    with pytest.raises(ValueError, match="planes"):
        qa.paged_evict(budget=4, max_seq_len=32, mass=None, key_positions=p["key_positions"], **c)
    with pytest.raises(ValueError, match="CUDA device"):
        qa.paged_evict(budget=4, max_seq_len=32, **c, **p)


# ---- the C ABI: fake addresses are never dereferenced, validation stops before any launch
FAKE = 0x10000


def c_cache(**over):
    from quantized_attention_mean_gb300._lib import SagePagedCache
    a = dict(k=FAKE, ks=(2 * 16 * 64, 16 * 64, 64), v=FAKE, vs=(2 * 16 * 64, 16 * 64, 64), pages=6, size=16, table=FAKE,
             ts=2, width=2, lens=FAKE, mass=FAKE, pos=FAKE)
    a.update(over)
    return SagePagedCache(a["k"], *a["ks"], a["v"], *a["vs"], a["pages"], a["size"], a["table"], a["ts"], a["width"],
                          a["lens"], a["mass"], a["pos"])


@pytest.fixture(scope="module")
def lib():
    from quantized_attention_mean_gb300 import _lib, build
    build.build()
    return _lib.load()


def attn(lib, c=None, **over):
    from quantized_attention_mean_gb300._lib import SagePacked
    a = dict(q=FAKE, batch=3, hq=4, hkv=2, maxn=32, d=64, dtype=0, layout=0, cap=0.0, ws=FAKE * 16, wsb=1 << 40)
    a.update(over)
    q = SagePacked(a["q"], 4 * 64, 64)
    c = c or c_cache()
    return lib.sage_paged_attn(ctypes.byref(q), ctypes.byref(c), ctypes.byref(q), None, None, None, a["batch"], a["hq"],
                               a["hkv"], a["maxn"], a["d"], a["dtype"], a["layout"], 0.0, a["cap"],
                               ctypes.c_void_p(a["ws"]), a["wsb"], None)


def test_c_attn_statuses(lib):
    assert attn(lib, d=129) == 2 and attn(lib, d=0) == 2
    assert attn(lib, dtype=2) == 3
    assert attn(lib, hq=3) == 5
    assert attn(lib, layout=2) == 1
    assert attn(lib, maxn=-1) == 1
    assert attn(lib, hkv=0) == 1
    assert attn(lib, cap=-1.0) == 1 and attn(lib, cap=float("nan")) == 1 and attn(lib, cap=float("inf")) == 1
    assert attn(lib, q=0) == 1 and attn(lib, q=FAKE + 1) == 4
    assert attn(lib, batch=0) == 0
    assert attn(lib, wsb=1024) == 6 and attn(lib, ws=0) == 6 and attn(lib, ws=FAKE * 16 + 8) == 6
    assert attn(lib, c_cache(k=FAKE + 1)) == 4
    assert attn(lib, c_cache(vs=(1, -1, 1))) == 4
    assert attn(lib, c_cache(size=0)) == 1 and attn(lib, c_cache(table=0)) == 1 and attn(lib, c_cache(lens=FAKE + 2)) == 1
    assert attn(lib, c_cache(size=65536, width=65536)) == 1      # slots past 32 bits
    assert lib.sage_paged_attn(None, None, None, None, None, None, 1, 1, 1, 1, 64, 0, 0, 0.0, 0.0, None, 0, None) == 1


def test_c_append_and_evict_statuses(lib):
    from quantized_attention_mean_gb300._lib import SagePacked
    t = SagePacked(FAKE, 128, 64)

    def append(c=None, cu=FAKE, batch=3, tokens=5, d=64, ws=0, wsb=0, k=t):
        c = c or c_cache()
        return lib.sage_paged_append(ctypes.byref(k), ctypes.byref(t), ctypes.byref(c), ctypes.c_void_p(cu), None, batch,
                                     tokens, 2, d, 0, 0, ctypes.c_void_p(ws), wsb, None)
    assert append(d=200) == 2
    assert append(cu=0) == 1
    assert append(tokens=-1) == 1
    assert append(tokens=0) == 0 and append(batch=0) == 0
    assert append(ws=FAKE * 16, wsb=128) == 6 and append(ws=FAKE * 16 + 4, wsb=1024) == 6
    assert append(k=SagePacked(FAKE + 1, 128, 64)) == 4 and append(k=SagePacked(FAKE, -128, 64)) == 4
    assert append(k=SagePacked(0, 128, 64)) == 1

    def evict(c=None, new=FAKE * 2, batch=3, maxn=32, budget=8, sink=0, recent=0, wsb=1 << 40):
        c = c or c_cache()
        return lib.sage_paged_evict(ctypes.byref(c), ctypes.c_void_p(new), batch, 2, maxn, 64, 0, 0, budget, sink, recent,
                                    ctypes.c_void_p(FAKE * 16), wsb, None)
    assert evict(budget=0) == 1 and evict(sink=5, recent=4) == 1 and evict(sink=-1) == 1
    assert evict(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == 1
    assert evict(new=0) == 1 and evict(new=FAKE) == 1             # none, and seq_lens itself
    assert evict(c_cache(mass=0)) == 1 and evict(c_cache(pos=0)) == 1
    assert evict(wsb=256) == 6
    assert evict(batch=0) == 0


def test_slots_and_lengths_at_the_ends(lib):
    assert attn(lib, c_cache(size=32768, width=65535)) == 1      # 2^31 - 32768 slots: the kernels look past the last
    assert attn(lib, c_cache(size=32768, width=65534), wsb=0) == 6
    t = c_cache()
    for new in (FAKE - 8, FAKE + 8):                             # three lengths that overlap the three of seq_lens
        assert lib.sage_paged_evict(ctypes.byref(t), ctypes.c_void_p(new), 3, 2, 32, 64, 0, 0, 8, 0, 0,
                                    ctypes.c_void_p(FAKE * 16), 1 << 40, None) == 1


def test_workspace_sizes(lib):
    assert qa.paged_attn_workspace_bytes(1, 3, 2, 10, 64) == 0
    assert qa.paged_attn_workspace_bytes(1, 4, 2, 10, 129) == 0
    plain, tracked = (qa.paged_attn_workspace_bytes(4, 8, 2, 1000, 128, m) for m in (False, True))
    assert tracked >= plain + 4 * 8 * 1000 * 4 > 0
    assert qa.paged_evict_workspace_bytes(4, 2, 100, 30) >= 4 * 2 * 30 * 8
    assert qa.paged_evict_workspace_bytes(4, 2, 100, -1) == 0
    assert lib.sage_status_string(13).decode().startswith("SAGE_ERR_PAGE")
