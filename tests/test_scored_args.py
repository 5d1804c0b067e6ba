"""What scored_attn refuses, on the CPU: the binding's checks and the C ABI's statuses (both come
before any device work)."""

import ctypes

import pytest
import torch

import quantized_attention_mean_gb300 as qa


def test_argument_checks():
    q, k = torch.zeros(1, 4, 64, 64, dtype=torch.float16), torch.zeros(1, 2, 80, 64, dtype=torch.float16)
    # (the checks of shapes, dtypes and devices that sage_attn makes come first)
    with pytest.raises(ValueError, match="v must have k's shape"):
        qa.scored_attn(q, k, k[:, :, :79])
    with pytest.raises(ValueError, match="CUDA device"):
        qa.scored_attn(q, k, k)


@pytest.fixture()
def on_cuda(monkeypatch):
    """The device checks out of the way, so that those behind them can be seen without a GPU."""
    from quantized_attention_mean_gb300 import scored
    monkeypatch.setattr(scored, "_check_dense_args", lambda *a: None)


def test_mask_checks(on_cuda):
    q, k = torch.zeros(1, 4, 64, 64, dtype=torch.float16), torch.zeros(1, 2, 80, 64, dtype=torch.float16)
    ids = torch.zeros(1, 64, dtype=torch.int32)
    with pytest.raises(ValueError, match="doc_ids_k needs doc_ids"):
        qa.scored_attn(q, k, k, doc_ids_k=torch.zeros(1, 80, dtype=torch.int32))
    with pytest.raises(ValueError, match="need doc_ids_k"):
        qa.scored_attn(q, k, k, doc_ids=ids)
    with pytest.raises(ValueError, match="doc_ids must"):
        qa.scored_attn(q, k, k, doc_ids=ids.long(), doc_ids_k=torch.zeros(1, 80, dtype=torch.int32))
    with pytest.raises(ValueError, match="doc_ids_k must"):
        qa.scored_attn(q, k, k, doc_ids=ids, doc_ids_k=ids)
    with pytest.raises(ValueError, match="prefix_lens needs is_causal"):
        qa.scored_attn(q, k, k, prefix_lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="prefix_lens must"):
        qa.scored_attn(q, k, k, is_causal=True, prefix_lens=torch.zeros(2, dtype=torch.int32))
    for offset in (2 ** 31, -2 ** 31):
        with pytest.raises(ValueError, match="q_offset"):
            qa.scored_attn(q, k, k, q_offset=offset)
    with pytest.raises(ValueError, match="slopes must"):
        qa.scored_attn(q, k, k, slopes=torch.zeros(2))


FAKE = 0x10000  # never dereferenced: validation stops before any launch


@pytest.fixture(scope="module")
def lib():
    from quantized_attention_mean_gb300 import _lib, build
    build.build()
    return _lib.load()


def call(lib, **over):
    from quantized_attention_mean_gb300._lib import SageTensor
    a = dict(q=FAKE, st=(2 * 256 * 64, 256 * 64, 64), lse=0, slopes=0, prefix=0, dq=0, dk=0, batch=1, hq=2, hkv=2, nq=256,
             nk=256, d=64, dtype=0, layout=0, causal=0, cap=0.0, offset=0, ret=0, ws=FAKE * 16, wsb=1 << 40)
    a.update(over)
    t = SageTensor(a["q"], (ctypes.c_int64 * 3)(*a["st"]))
    ok = SageTensor(FAKE, (ctypes.c_int64 * 3)(2 * 256 * 64, 256 * 64, 64))
    r = ctypes.byref
    return lib.sage_scored_attn(r(t), r(ok), r(ok), r(ok), a["lse"], a["slopes"], a["prefix"], a["dq"], a["dk"], a["batch"],
                                a["hq"], a["hkv"], a["nq"], a["nk"], a["d"], a["dtype"], a["layout"], a["causal"], 0.0,
                                a["cap"], a["offset"], a["ret"], a["ws"], a["wsb"], None)


def test_c_statuses(lib):
    assert call(lib, d=0) == 2 and call(lib, d=129) == 2
    assert call(lib, dtype=2) == 3
    assert call(lib, layout=2) == 1
    assert call(lib, hq=3) == 5
    assert call(lib, hq=0) == 1 and call(lib, hkv=0) == 1 and call(lib, nq=-1) == 1 and call(lib, nk=-1) == 1
    for cap in (-1.0, float("nan"), float("inf"), 4097.0, 1e-39):
        assert call(lib, cap=cap) == 1
    assert call(lib, ret=1) == 1                          # return_lse without an lse buffer
    assert call(lib, prefix=FAKE) == 1                    # a prefix without a causal mask
    assert call(lib, dq=FAKE) == 1 and call(lib, dk=FAKE) == 1
    assert call(lib, slopes=FAKE + 2) == 1
    assert call(lib, q=0) == 1 and call(lib, q=FAKE + 1) == 4 and call(lib, st=(64, -64, 64)) == 4
    assert call(lib, offset=2 ** 31 - 1) == 1 and call(lib, offset=-2 ** 31) == 1
    assert call(lib, nq=0) == 0 and call(lib, batch=0) == 0
    assert call(lib, dq=FAKE, dk=FAKE, wsb=256) == 6 and call(lib, dq=FAKE, dk=FAKE, ws=0) == 6
    assert call(lib, ws=FAKE * 16 + 16) == 6 and call(lib, wsb=128) == 6
    assert call(lib, nq=2, nk=4096, ws=0) == 6                  # split over the keys
    assert lib.sage_scored_attn_workspace_size(1, 2, 2, 256, 256, 64, 3) == 256     # no documents: the status word alone
    # a query tensor that needs a copy needs the larger workspace
    small = lib.sage_scored_attn_workspace_size(1, 2, 2, 256, 256, 64, 1)
    assert call(lib, st=(2 * 256 * 64, 256 * 64, 65), wsb=small) == 6
    assert lib.sage_scored_attn(None, None, None, None, 0, 0, 0, 0, 0, 1, 1, 1, 1, 1, 64, 0, 0, 0, 0.0, 0.0, 0, 0, None, 0,
                                None) == 1


def test_workspace_sizes():
    assert qa.scored_attn_workspace_bytes(1, 3, 2, 10, 10, 64) == 0
    assert qa.scored_attn_workspace_bytes(1, 4, 2, 10, 10, 200) == 0
    a, b = (qa.scored_attn_workspace_bytes(2, 4, 2, 1000, 1000, 72, p) for p in (True, False))
    assert b >= a + 2 * (4 + 2 * 2) * 1000 * 128 * 2
