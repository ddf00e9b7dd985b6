"""Refusals of the calls of q1_memory.h (no GPU needed): invalid arguments get a
status and a message before any HIP call; empty calls are no-ops."""
import ctypes
import os

import pytest

from gemm_decode_q1_amd import memory as D
from gemm_decode_q1_amd import q1 as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libq1.so not built")

FAKE = 0x10000  # never dereferenced: validation fails first
BIG = 1 << 40


def said():
    return B.load_library().q1_last_error().decode()


def kv(**kw):
    d = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, pages=10, page_size=16, Hkv=2, D=128, bits=4, reserved=0)
    d.update(kw)
    return ctypes.byref(D._KV(**d))


KV_BAD = [
    (dict(bits=3), -2, "bits"), (dict(D=96), -2, "D must be"), (dict(Hkv=0), -1, "Hkv"), (dict(Hkv=5000), -2, "heads"),
    (dict(pages=-1), -1, "pages"), (dict(page_size=0), -1, "page_size"), (dict(reserved=1), -1, "reserved"),
    (dict(pages=1 << 20, page_size=1 << 20), -2, "too large"), (dict(page_size=1 << 25), -2, "too large"),
    (dict(k=None), -1, "NULL"), (dict(v_scales=None), -1, "NULL"), (dict(v=FAKE + 8), -1, "16-byte"),
    (dict(k_scales=FAKE + 4), -1, "8-byte"),
]


def write(c, k=FAKE, v=FAKE, dtype=B.Q1_BF16, k_ld=256, v_ld=256, tokens=3, slots=FAKE):
    return B.load_library().q1_kv_write(c, k, v, dtype, k_ld, v_ld, tokens, slots, None)


def read(c, slots=FAKE, rows=3, k=FAKE, v=FAKE, dtype=B.Q1_BF16):
    return B.load_library().q1_kv_read(c, slots, rows, k, v, dtype, None)


def query(**kw):
    d = dict(q=FAKE, page_table=FAKE, lens=FAKE, out=FAKE, lse=FAKE, q_ld=8 * 128, B=2, T=1, max_pages=3, Hq=8,
             dtype=B.Q1_BF16, out_dtype=B.Q1_BF16, scale=1.0)
    d.update(kw)
    return ctypes.byref(D._KVQuery(**d))


@pytest.mark.parametrize("kw,code,msg", KV_BAD)
def test_pages(kw, code, msg):
    c = kv(**kw)
    for call in (lambda: write(c), lambda: read(c), lambda: B.load_library().q1_kv_attn(c, query(), None, 0, None)):
        assert call() == code and msg in said()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(tokens=-1), -1, "tokens"), (dict(tokens=BIG), -2, "too large"),
    (dict(k=None), -1, "NULL"), (dict(slots=None), -1, "NULL"), (dict(v=FAKE + 2), -1, "16-byte"),
    (dict(slots=FAKE + 2), -1, "4-byte"), (dict(k_ld=128), -1, "cover"), (dict(v_ld=260), -1, "multiples of 8"),
    (dict(k_ld=1 << 23), -2, "2^23"),
])
def test_write(kw, code, msg):
    assert write(kv(), **kw) == code and msg in said()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=7), -1, "out dtype"), (dict(rows=-1), -1, "rows"), (dict(rows=BIG), -2, "too large"),
    (dict(k=None), -1, "NULL"), (dict(slots=None), -1, "NULL"), (dict(v=FAKE + 2), -1, "16-byte"),
    (dict(slots=FAKE + 2), -1, "4-byte"),
])
def test_read(kw, code, msg):
    assert read(kv(), **kw) == code and msg in said()


def test_empty_writes_and_reads():
    assert write(kv(), tokens=0, k=None, v=None, slots=None) == 0
    assert read(kv(), rows=0, k=None, v=None, slots=None) == 0
    assert write(None) == -1 and read(None) == -1 and "NULL" in said()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(out_dtype=9), -1, "out dtype"), (dict(Hq=7), -1, "multiple"),
    (dict(Hq=0), -1, "multiple"), (dict(Hq=8192, q_ld=8192 * 128), -2, "too many heads"), (dict(B=-1), -1, ">= 0"),
    (dict(T=-1), -1, ">= 0"), (dict(max_pages=-1), -1, ">= 0"), (dict(q_ld=1000), -1, "cover"),
    (dict(q_ld=1028), -1, "multiple of 8"), (dict(max_pages=1 << 30), -2, "too large"), (dict(B=1 << 20, T=1 << 20), -2, "too large"),
    (dict(B=1 << 26), -2, "too large"), (dict(q=None), -1, "NULL"), (dict(out=None), -1, "NULL"), (dict(lens=None), -1, "NULL"),
    (dict(page_table=None), -1, "NULL"), (dict(q=FAKE + 8), -1, "16-byte"), (dict(lse=FAKE + 2), -1, "4-byte"),
])
def test_attention(kw, code, msg):
    L = B.load_library()
    assert L.q1_kv_attn(kv(), query(**kw), FAKE, 1 << 40, None) == code and msg in said()


def test_attention_empty_and_workspace():
    L = B.load_library()
    assert L.q1_kv_attn(kv(), None, None, 0, None) == -1 and L.q1_kv_attn_workspace_bytes(kv(), None) == 0
    assert L.q1_kv_attn(kv(), query(B=0), None, 0, None) == 0 and L.q1_kv_attn(kv(), query(T=0), None, 0, None) == 0
    c, a = kv(pages=1000), query(max_pages=500)
    need = L.q1_kv_attn_workspace_bytes(c, a)
    assert need > 0
    assert L.q1_kv_attn(c, a, FAKE, need - 1, None) == -3
    assert L.q1_kv_attn(c, a, None, need, None) == -3
    assert L.q1_kv_attn(c, a, FAKE + 64, need, None) == -1 and "256-byte" in said()


def conv(**kw):
    d = dict(x=FAKE, weight=FAKE, bias=None, state=FAKE, slot_ids=None, out=FAKE, x_ld=64, slots=4, C=64, W=4,
             dtype=B.Q1_BF16, silu=1, reserved=0)
    d.update(kw)
    return ctypes.byref(D._Conv(**d))


CONV_BAD = [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(reserved=1), -1, "reserved"), (dict(W=1), -2, "W must be"),
    (dict(W=5), -2, "W must be"), (dict(C=60), -1, "multiple of 8"), (dict(C=0), -1, "multiple of 8"),
    (dict(C=1 << 21, x_ld=1 << 21), -2, "2^20"), (dict(silu=2), -1, "silu"), (dict(x=None), -1, "NULL"),
    (dict(weight=None), -1, "NULL"), (dict(state=None), -1, "NULL"), (dict(out=None), -1, "NULL"),
    (dict(bias=FAKE + 8), -1, "16-byte"), (dict(x=FAKE + 8), -1, "16-byte"), (dict(slot_ids=FAKE + 1), -1, "4-byte"),
    (dict(slots=0), -1, "slots"), (dict(slots=2), -1, "as many state slots"), (dict(x_ld=56), -1, "cover"),
    (dict(x_ld=68), -1, "multiples of 8"), (dict(x_ld=1 << 23), -2, "2^23"), (dict(slots=BIG), -2, "too large"),
]


@pytest.mark.parametrize("kw,code,msg", CONV_BAD)
def test_conv(kw, code, msg):
    L = B.load_library()
    assert L.q1_conv_step(conv(**kw), 3, 1, None) == code and msg in said()
    assert L.q1_conv_prefill(conv(**kw), 10, 3, FAKE, None) == code and msg in said()


def scan(**kw):
    d = dict(x=FAKE, dt=FAKE, B=FAKE, C=FAKE, z=FAKE, A=FAKE, D=FAKE, dt_bias=FAKE, state=FAKE, slot_ids=None, out=FAKE,
             x_ld=64, dt_ld=64, b_ld=16, c_ld=16, z_ld=64, slots=4, Di=64, N=16, dtype=B.Q1_BF16, dt_dtype=B.Q1_BF16,
             out_dtype=B.Q1_BF16, softplus=1, reserved=0)
    d.update(kw)
    return ctypes.byref(D._Scan(**d))


SCAN_BAD = [
    (dict(dtype=B.Q1_F32), -2, "bf16 or fp16"), (dict(reserved=1), -1, "reserved"), (dict(dt_dtype=B.Q1_F16), -2, "dt must"),
    (dict(out_dtype=5), -1, "out dtype"), (dict(N=12), -2, "N must be"), (dict(Di=60), -1, "multiple of 8"),
    (dict(Di=1 << 19, x_ld=1 << 19), -2, "2^18"), (dict(softplus=2), -1, "softplus"), (dict(x=None), -1, "NULL"),
    (dict(dt=None), -1, "NULL"), (dict(B=None), -1, "NULL"), (dict(C=None), -1, "NULL"), (dict(A=None), -1, "NULL"),
    (dict(state=None), -1, "NULL"), (dict(out=None), -1, "NULL"), (dict(B=FAKE + 8), -1, "16-byte"),
    (dict(z=FAKE + 8), -1, "16-byte"), (dict(D=FAKE + 2), -1, "4-byte"), (dict(slots=0), -1, "slots"),
    (dict(slots=2), -1, "as many state slots"), (dict(b_ld=8), -1, "cover"), (dict(z_ld=0), -1, "cover"),
    (dict(dt_ld=68), -1, "multiples of 8"), (dict(c_ld=1 << 23), -2, "2^23"), (dict(slots=BIG), -2, "too large"),
]


@pytest.mark.parametrize("kw,code,msg", SCAN_BAD)
def test_scan(kw, code, msg):
    L = B.load_library()
    assert L.q1_scan_step(scan(**kw), 3, 1, None) == code and msg in said()
    assert L.q1_scan_prefill(scan(**kw), 10, 3, FAKE, None, 0, None) == code and msg in said()


@pytest.mark.parametrize("what", ["conv", "scan"])
def test_counts(what):
    L = B.load_library()
    d = conv() if what == "conv" else scan()
    step = L.q1_conv_step if what == "conv" else L.q1_scan_step

    def prefill(d, tokens, nseq, cu):
        if what == "conv":
            return L.q1_conv_prefill(d, tokens, nseq, cu, None)
        return L.q1_scan_prefill(d, tokens, nseq, cu, None, 0, None)

    assert step(None, 1, 1, None) == -1 and prefill(None, 1, 1, FAKE) == -1
    assert step(d, -1, 1, None) == -1 and step(d, 1, -1, None) == -1
    assert step(d, 0, 1, None) == 0 and step(d, 2, 0, None) == 0
    assert step(d, 1 << 20, 1 << 20, None) == -2
    assert prefill(d, -1, 1, FAKE) == -1 and prefill(d, 0, 3, FAKE) == 0 and prefill(d, 10, 0, FAKE) == 0
    assert prefill(d, 10, 1, None) == -1 and "cu_seqlens" in said()
    assert prefill(d, 10, 1, FAKE + 2) == -1 and prefill(d, 1 << 31, 1, FAKE) == -2


def test_scan_without_gate_needs_no_stride():
    L = B.load_library()
    need = L.q1_scan_prefill_workspace_bytes(scan(z=None, z_ld=0), 5000, 1)
    assert need > 0
    d = scan(z=None, z_ld=0)
    assert L.q1_scan_prefill(d, 5000, 1, FAKE, None, 0, None) == -3
    assert L.q1_scan_prefill(d, 5000, 1, FAKE, FAKE, need - 1, None) == -3
    assert L.q1_scan_prefill(d, 5000, 1, FAKE, FAKE + 128, need, None) == -1 and "256-byte" in said()
    assert L.q1_scan_prefill_workspace_bytes(scan(N=12), 100, 1) == 0 and "N must be" in said()
    assert L.q1_scan_prefill_workspace_bytes(d, -1, 1) == 0 and L.q1_scan_prefill_workspace_bytes(d, 1 << 31, 1) == 0


@pytest.mark.parametrize("page_size,pages_", [(1, (1 << 31) - 1), (1, (1 << 31) - (1 << 16) + 1), (16, 1 << 27), (1 << 16, (1 << 15) - 1)])
def test_tokens_of_a_sequence(page_size, pages_):
    """A table may have room for 2^31 - 2^16 tokens: the kernels count the tile behind the last one in 31 bits."""
    c = kv(pages=3, page_size=page_size, Hkv=1)
    room = page_size * pages_
    L = B.load_library()
    status = L.q1_kv_attn(c, query(B=1, max_pages=pages_, q=None), None, 0, None)
    if room > (1 << 31) - (1 << 16):
        assert status == -2 and "too large" in said()
    else:
        assert status == -1 and "NULL" in said()
