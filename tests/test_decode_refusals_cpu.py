"""Refusals of the decode-step operators (no GPU needed): invalid arguments get
a status and a message before any HIP call; empty calls are no-ops."""
import ctypes
import os

import pytest

from gemm_decode_q1_amd import decode as D
from gemm_decode_q1_amd import q1 as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libq1.so not built")

FAKE = 0x10000  # never dereferenced: validation fails first


def delta(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_ld=2 * 128, k_ld=2 * 128, v_ld=6 * 128, g=FAKE, beta=FAKE, state=FAKE,
             slot_ids=None, out=FAKE, slots=4, Hk=2, Hv=6, Dk=128, Dv=128, dtype=B.Q1_BF16, out_dtype=B.Q1_BF16,
             l2norm=1, scale=1.0)
    d.update(kw)
    return D._Delta(**d)


def said():
    return B.load_library().q1_last_error().decode()


DELTA_BAD = [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(out_dtype=5), -1, "out dtype"),
    (dict(Hk=0), -1, "multiple of key heads"), (dict(Hv=5), -1, "multiple of key heads"),
    (dict(Dk=96), -2, "Dk must be"), (dict(Dv=24), -2, "Dv must be"), (dict(Dv=272), -2, "Dv must be"),
    (dict(l2norm=2), -1, "l2norm"), (dict(q=None), -1, "NULL"), (dict(state=None), -1, "NULL"),
    (dict(beta=None), -1, "NULL"), (dict(k=FAKE + 8), -1, "16-byte"), (dict(out=FAKE + 8), -1, "16-byte"),
    (dict(g=FAKE + 2), -1, "4-byte"), (dict(slot_ids=FAKE + 1), -1, "4-byte"), (dict(q_ld=128), -1, "row strides"),
    (dict(v_ld=6 * 128 + 4), -1, "multiples of 8"), (dict(slots=0), -1, "slots must be positive"),
    (dict(slots=2), -1, "as many state slots"), (dict(Hk=1, Hv=8192), -2, "too many heads"),
    (dict(slots=1 << 40), -2, "too large"),
]


@pytest.mark.parametrize("kw,code,msg", DELTA_BAD)
def test_delta_refusals(kw, code, msg):
    L, d = B.load_library(), delta(**kw)
    assert L.q1_delta_step(ctypes.byref(d), 3, 1, None) == code and msg in said()
    assert L.q1_delta_prefill(ctypes.byref(d), 70, 3, FAKE, None, 0, None) == code and msg in said()


def test_delta_counts():
    L, d = B.load_library(), delta()
    assert L.q1_delta_step(None, 1, 1, None) == -1
    assert L.q1_delta_step(ctypes.byref(d), -1, 1, None) == -1
    assert L.q1_delta_step(ctypes.byref(d), 1, -1, None) == -1
    assert L.q1_delta_step(ctypes.byref(d), 0, 1, None) == 0
    assert L.q1_delta_step(ctypes.byref(d), 2, 0, None) == 0
    assert L.q1_delta_step(ctypes.byref(d), 1 << 20, 1 << 20, None) == -2
    assert L.q1_delta_prefill(ctypes.byref(d), -1, 1, FAKE, None, 0, None) == -1
    assert L.q1_delta_prefill(ctypes.byref(d), 0, 3, FAKE, None, 0, None) == 0
    assert L.q1_delta_prefill(ctypes.byref(d), 10, 0, FAKE, None, 0, None) == 0
    assert L.q1_delta_prefill(ctypes.byref(d), 10, 1, None, None, 0, None) == -1 and "cu_seqlens" in said()


def test_delta_prefill_workspace():
    L, d = B.load_library(), delta()
    assert L.q1_delta_prefill_workspace_bytes(ctypes.byref(delta(Dk=32)), 100, 1) == 0 and "Dk" in said()
    need = L.q1_delta_prefill_workspace_bytes(ctypes.byref(d), 100, 3)
    if need:
        assert L.q1_delta_prefill(ctypes.byref(d), 100, 3, FAKE, None, 0, None) == -3
        assert L.q1_delta_prefill(ctypes.byref(d), 100, 3, FAKE, FAKE, need - 1, None) == -3
        assert L.q1_delta_prefill(ctypes.byref(d), 100, 3, FAKE, FAKE + 128, need, None) == -1


def attn(**kw):
    d = dict(q=FAKE, k_prefix=FAKE, v_prefix=FAKE, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, suffix_lens=FAKE,
             out=FAKE, lse=FAKE, q_ld=8 * 128, prefix_ld=2 * 128, B=2, P=10, pages=4, max_pages=2, page_size=16, Hq=8,
             Hkv=2, D=128, dtype=B.Q1_BF16, out_dtype=B.Q1_BF16, scale=1.0)
    d.update(kw)
    return D._Attn(**d)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(out_dtype=9), -1, "out dtype"),
    (dict(Hkv=3), -1, "multiple of key/value heads"), (dict(Hq=0), -1, "multiple of key/value heads"),
    (dict(D=96), -2, "D must be"), (dict(B=-1), -1, ">= 0"), (dict(P=-1), -1, ">= 0"), (dict(pages=-1), -1, ">= 0"),
    (dict(page_size=0), -1, "page_size"), (dict(prefix_ld=128), -1, "prefix_ld"), (dict(q_ld=128), -1, "q_ld"),
    (dict(q_ld=1028), -1, "multiples of 8"), (dict(q=None), -1, "NULL"), (dict(out=None), -1, "NULL"),
    (dict(k_prefix=None), -1, "NULL"), (dict(v_pages=None), -1, "NULL"), (dict(page_table=None), -1, "NULL"),
    (dict(suffix_lens=None), -1, "NULL"), (dict(k_pages=FAKE + 8), -1, "16-byte"), (dict(q=FAKE + 2), -1, "16-byte"),
    (dict(lse=FAKE + 2), -1, "4-byte"), (dict(max_pages=1 << 30, page_size=64), -2, "too large"),
    (dict(P=1 << 40), -2, "too large"), (dict(Hq=8192, Hkv=2, q_ld=8192 * 128), -2, "too many heads"),
])
def test_attn_refusals(kw, code, msg):
    L, a = B.load_library(), attn(**kw)
    assert L.q1_prefix_attn(ctypes.byref(a), None, 0, None) == code and msg in said()


def test_attn_empty_and_workspace():
    L = B.load_library()
    assert L.q1_prefix_attn(None, None, 0, None) == -1
    assert L.q1_prefix_attn(ctypes.byref(attn(B=0)), None, 0, None) == 0
    a = attn(P=5000)
    need = L.q1_prefix_attn_workspace_bytes(ctypes.byref(a))
    if need:
        assert L.q1_prefix_attn(ctypes.byref(a), FAKE, need - 1, None) == -3
        assert L.q1_prefix_attn(ctypes.byref(a), FAKE + 64, need, None) == -1


def sample(logits=FAKE, dtype=B.Q1_F32, b=2, v=100, ld=100, u=FAKE, t=None, k=None, p=None, m=None, tok=FAKE, i64=1,
           lp=FAKE, ws=None, n=0):
    return B.load_library().q1_sample(logits, dtype, b, v, ld, u, t, k, p, m, tok, i64, lp, ws, n, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=7), -1, "logits must be"), (dict(b=-1), -1, "B must be"), (dict(v=0), -1, "V must be"),
    (dict(v=(1 << 22) + 1, ld=1 << 23), -2, "2^22"), (dict(ld=99), -1, "row stride"), (dict(i64=2), -1, "tokens_are_int64"),
    (dict(logits=None), -1, "NULL"), (dict(u=None), -1, "NULL"), (dict(tok=None), -1, "NULL"),
    (dict(logits=FAKE + 2), -1, "misaligned"), (dict(tok=FAKE + 4), -1, "aligned"), (dict(t=FAKE + 2), -1, "aligned"),
    (dict(b=1 << 21), -2, "too large"),
])
def test_sample_refusals(kw, code, msg):
    assert sample(**kw) == code and msg in said()


def test_sample_empty_and_workspace():
    assert sample(b=0) == 0
    L = B.load_library()
    assert L.q1_sample_workspace_bytes(-1, 5) == 0 and "B must" in said()
    need = L.q1_sample_workspace_bytes(2, 100)
    if need:
        assert sample() == -3
        assert sample(ws=FAKE, n=need - 1) == -3
        assert sample(ws=FAKE + 32, n=need) == -1


@pytest.mark.parametrize("kw", [dict(q_ld=1 << 23), dict(k_ld=1 << 23), dict(v_ld=1 << 24)])
def test_delta_stride_limit(kw):
    L, d = B.load_library(), delta(**kw)
    assert L.q1_delta_step(ctypes.byref(d), 3, 1, None) == -2 and "2^23" in said()
    assert L.q1_delta_prefill(ctypes.byref(d), 70, 3, FAKE, None, 0, None) == -2 and "2^23" in said()


@pytest.mark.parametrize("kw,msg", [(dict(prefix_ld=1 << 23), "2^23"), (dict(pages=1 << 27), "too large"),
                                    (dict(P=1 << 31), "too large")])
def test_attn_limits(kw, msg):
    L, a = B.load_library(), attn(**kw)
    assert L.q1_prefix_attn(ctypes.byref(a), None, 0, None) == -2 and msg in said()
