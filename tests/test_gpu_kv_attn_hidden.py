"""Attention over quantised pages where a value that some queries do not see stands for no
finite number: the NaN code of E4M3 under an ordinary scale, and scales that carry a code
past bf16's range.  `q1_kv_write` makes neither, but a program may bring pages of its own.
The queries that do not see the token have the same bits as without it; the others lose its
column, and no column of another block."""
import pytest
import torch

from test_gpu_kv_attn import Case
from test_gpu_kv_attn_rows import Prompts

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q

# bits, scale byte, code of the element (4 bits: one of two in the byte)
ODD = [(8, 127, 0x7f), (8, 127, 0xff), (8, 250, 0x7e), (8, 254, 0xfe), (4, 253, 0x7), (4, 254, 0xf), (4, 254, 0x4)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    yield
    torch.cuda.synchronize()


def plant(cache, page, head, row, i, byte, code):
    """Element i of a value row gets the code, and its block the scale byte."""
    if cache.bits == 8:
        cache.v[page, head, row, i] = code
    else:
        old = int(cache.v[page, head, row, i // 2])
        cache.v[page, head, row, i // 2] = old & 0xf0 | code if i % 2 == 0 else old & 0x0f | code << 4
    cache.v_scales[page, head, row, i // 32] = byte


def compare(out, lse, clean, at, head, heads, i, byte):
    """`at`: the first query that sees the token; `heads`: query heads of its key/value head."""
    block = slice(i // 32 * 32, i // 32 * 32 + 32)
    assert torch.equal(lse, clean[1])
    if byte != 127:  # (else the block's other values are as they were)
        assert not torch.equal(out[:, at:, heads, block], clean[0][:, at:, heads, block])
    else:
        assert out[:, at:, heads, i].isnan().all()
    other = out.clone()
    other[:, at:, heads, block] = clean[0][:, at:, heads, block]
    assert torch.equal(other, clean[0])


@pytest.mark.parametrize("bits,byte,code", ODD)
@pytest.mark.parametrize("Hq,Hkv,D,T,n,dt", [(4, 2, 64, 3, 40, "bf16"), (6, 1, 128, 4, 200, "f16"), (8, 2, 256, 2, 130, "bf16"),
                                             (40, 1, 64, 2, 96, "f16"), (12, 1, 128, 5, 6, "bf16"), (4, 2, 256, 9, 6000, "bf16")])
def test_few_queries(Hq, Hkv, D, T, n, dt, bits, byte, code):
    c = Case(T + n, 1, T, Hq, Hkv, D, [n], 16, bits, dt)
    head, heads = Hkv - 1, slice((Hkv - 1) * (Hq // Hkv), Hq)
    clean = [x.clone() for x in c.run(out_dtype=torch.float32)]
    assert torch.isfinite(clean[0]).all()
    for back, i in ((0, D - 1), (1, 0), (0, D // 2 + 9)):  # the last token, which one query sees, and the one before
        at = n - 1 - back
        page, row = c.table[0, at // 16], at % 16
        kept = c.cache.v[page, head, row].clone(), c.cache.v_scales[page, head, row].clone()
        plant(c.cache, page, head, row, i, byte, code)
        out, lse = c.run(out_dtype=torch.float32)
        compare(out, lse, clean, T - 1 - back, head, heads, i, byte)
        c.cache.v[page, head, row], c.cache.v_scales[page, head, row] = kept


@pytest.mark.parametrize("bits,byte,code", ODD)
@pytest.mark.parametrize("D,Hkv,dt", [(64, 32, "bf16"), (128, 32, "f16"), (256, 16, "bf16")])
def test_prompts(D, Hkv, dt, bits, byte, code):
    T = n = 1024
    c = Prompts(D + bits, 1, T, Hkv, Hkv, D, [n], 64, bits, dt)
    clean = [x.clone() for x in c.run(out_dtype=torch.float32)]
    for at, i in ((777, D - 1), (1023, 0), (512, D // 2 + 17)):
        page, row = c.table[0, at // 64], at % 64
        kept = c.cache.v[page, 3, row].clone(), c.cache.v_scales[page, 3, row].clone()
        plant(c.cache, page, 3, row, i, byte, code)
        out, lse = c.run(out_dtype=torch.float32)
        compare(out, lse, clean, at, 3, slice(3, 4), i, byte)
        c.cache.v[page, 3, row], c.cache.v_scales[page, 3, row] = kept


@pytest.mark.parametrize("byte,code", [(127, 0x7f), (254, 0xfe)])
def test_keys(byte, code):
    """The same of a key: queries that do not see it have their bits."""
    c = Case(5, 1, 4, 6, 1, 128, [200], 16, 8, "bf16")
    clean = [x.clone() for x in c.run(out_dtype=torch.float32)]
    page, row = c.table[0, 199 // 16], 199 % 16
    c.cache.k[page, 0, row, 5], c.cache.k_scales[page, 0, row, 0] = code, byte
    out, lse = c.run(out_dtype=torch.float32)
    assert torch.equal(out[:, :3], clean[0][:, :3]) and torch.equal(lse[:, :3], clean[1][:, :3])
    if byte == 127:
        assert out[:, 3].isnan().all() and lse[:, 3].isnan().all()
