"""What the binding of decoder memory checks of its operands and keeps, on host tensors
(no GPU needed: the device check is taken out, and a stand-in takes the calls)."""
import pytest
import torch

from gemm_decode_q1_amd import decode as D
from gemm_decode_q1_amd import memory as M


class Library:
    """Stands in for the library: takes any call, wants 4096 bytes of workspace."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *args: 4096
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture(autouse=True)
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(D, "_same_device", lambda first, **others: None)
    monkeypatch.setattr(M, "_same_device", lambda first, **others: None)
    monkeypatch.setattr(D, "_stream_of", lambda index: 0)
    monkeypatch.setattr(D, "_device", lambda: -1)
    monkeypatch.setattr(M, "load_library", lambda: lib)
    for kept in ("_write_layouts", "_read_layouts", "_kv_layouts", "_conv_layouts", "_scan_layouts", "_scan_needs"):
        monkeypatch.setattr(M, kept, {})
    return lib


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32)


def cache(bits=4, D=64, pages=3, page=5, Hkv=2):
    return M.PackedKV.empty(pages, page, Hkv, D, bits, device="cpu")


@pytest.mark.parametrize("bits,D", [(4, 64), (8, 64), (4, 128), (8, 256)])
def test_pages_know_their_geometry(bits, D):
    c = cache(bits, D)
    assert (c.bits, c.D, c.pages, c.page_size, c.Hkv) == (bits, D, 3, 5, 2)
    assert c.k.shape == (3, 2, 5, D * bits // 8) and c.v_scales.shape == (3, 2, 5, D // 32)
    again = M.PackedKV(c.k, c.v, c.k_scales, c.v_scales, bits)
    assert again._desc == c._desc


def test_pages_are_checked():
    c = cache()
    t = [c.k, c.v, c.k_scales, c.v_scales]
    for bits in (2, 16, 0):
        with pytest.raises(ValueError, match="bits"):
            M.PackedKV(*t, bits)
    for i, odd in ((0, c.k[0]), (0, c.k.float()), (1, c.v[:2]), (1, c.v[..., ::2]), (2, c.k_scales[..., :1]), (3, c.v_scales.int()),
                   (0, c.k.transpose(1, 2)), (2, c.k_scales[:, :, :4])):
        given = list(t)
        given[i] = odd
        with pytest.raises(ValueError):
            M.PackedKV(*given, 4)
    with pytest.raises(ValueError, match="D must be"):
        M.PackedKV(*(z(3, 2, 5, w, dtype=torch.uint8) for w in (48, 48, 3, 3)), 4)


def attn(c, q=None, table=None, lens=None, **kw):
    return M.q1_kv_attn(z(2, 3, 4, 64) if q is None else q, c, i32(0, 1, 2, 0).view(2, 2) if table is None else table,
                        i32(3, 4) if lens is None else lens, **kw)


def scan(x=None, **kw):
    given = dict(x=z(9, 16), dt=z(9, 16), A=z(16, 8, dtype=torch.float32), B=z(9, 8), C=z(9, 8),
                 state=z(2, 16, 8, dtype=torch.float32), cu_seqlens=i32(0, 4, 9))
    given.update(kw)
    if x is not None:
        given["x"] = x
    return M.q1_scan_prefill(**given)


def test_outputs_and_layouts_kept(library, monkeypatch):
    """The second call of a layout is not checked again, one of another layout is; nothing is
    kept of the tensors themselves."""
    monkeypatch.setattr(D, "_workspace", lambda nbytes, index, stream: z(nbytes, dtype=torch.uint8))
    c = cache()
    for _ in range(2):
        out, lse = attn(c)
        assert out.shape == (2, 3, 4, 64) and out.dtype == torch.bfloat16 and lse.shape == (2, 3, 4)
    assert len(M._kv_layouts) == 1
    wide = z(2, 3, 6, 64)
    out, _ = attn(c, q=wide[:, :, :4])
    assert len(M._kv_layouts) == 2 and out.is_contiguous()
    first, second = (call[1][1] for call in library.calls[1:3])
    assert first != second  # another row stride
    out, _ = attn(c, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    given = z(2, 3, 4, 64, dtype=torch.float16)
    assert attn(c, out=given)[0] is given
    x = z(9, 16)
    for _ in range(2):
        assert scan(x).shape == (9, 16)
    assert len(M._scan_layouts) == 1 and len(M._scan_needs) == 1
    assert M.q1_scan_step(z(2, 1, 16), z(2, 1, 16), z(16, 8, dtype=torch.float32), z(2, 1, 8), z(2, 1, 8),
                          z(2, 16, 8, dtype=torch.float32), out_dtype=torch.float32).dtype == torch.float32


@pytest.mark.parametrize("kw", [dict(q=z(2, 4, 64)), dict(q=z(2, 3, 4, 128)), dict(table=i32(0, 1)), dict(table=z(2, 2)),
                                dict(lens=i32(1)), dict(lens=z(2)), dict(table=i32(0, 1, 2, 0).view(2, 2).t()),
                                dict(q=z(2, 4, 3, 64).transpose(1, 2)), dict(out=z(2, 3, 4, 32)), dict(lse=z(2, 3, 4)),
                                dict(out=z(2, 3, 4, 64), out_dtype=torch.float32),
                                dict(workspace=z(4096)), dict(workspace=z(8192, dtype=torch.uint8)[::2])])
def test_attention_refuses(library, kw):
    with pytest.raises(ValueError):
        attn(cache(), **kw)
    assert not library.calls


@pytest.mark.parametrize("kw", [dict(x=z(9)), dict(dt=z(9, 8)), dict(A=z(16, 8)), dict(A=z(8, 16, dtype=torch.float32).t()),
                                dict(B=z(9, 16)), dict(C=z(9, 8, dtype=torch.float16)), dict(state=z(2, 16, 16, dtype=torch.float32)),
                                dict(cu_seqlens=torch.tensor([0, 9])), dict(cu_seqlens=i32()), dict(slots=i32(1)),
                                dict(z=z(8, 16)), dict(D=z(16)), dict(dt_bias=z(8, dtype=torch.float32)),
                                dict(out=z(9, 16, dtype=torch.float16), out_dtype=torch.float32), dict(workspace=z(4096))])
def test_scan_refuses(library, kw):
    with pytest.raises(ValueError):
        scan(**kw)
    assert not library.calls


@pytest.mark.parametrize("kw", [dict(x=z(9)), dict(weight=z(16)), dict(weight=z(8, 4)), dict(weight=z(16, 4, dtype=torch.float16)),
                                dict(state=z(2, 4, 16)), dict(state=z(2, 3, 16, dtype=torch.float32)), dict(bias=z(8)),
                                dict(slots=i32(0, 1, 2)), dict(out=z(9, 16, dtype=torch.float32)), dict(cu_seqlens=z(3)),
                                dict(x=z(16, 9).t())])
def test_convolution_refuses(library, kw):
    given = dict(x=z(9, 16), weight=z(16, 4), state=z(2, 3, 16), cu_seqlens=i32(0, 4, 9))
    assert M.q1_conv_prefill(**given).shape == (9, 16)
    given.update(kw)
    with pytest.raises(ValueError):
        M.q1_conv_prefill(**given)
    assert len(library.calls) == 1


@pytest.mark.parametrize("kw", [dict(k=z(7, 2, 32)), dict(v=z(6, 2, 64)), dict(v=z(7, 2, 64, dtype=torch.float16)),
                                dict(slots=i32(*range(7)).long()), dict(slots=i32(*range(14))[::2]), dict(k=z(7, 64, 2).transpose(1, 2))])
def test_write_refuses(library, kw):
    given = dict(k=z(7, 2, 64), v=z(7, 2, 64), slots=i32(*range(7)))
    M.q1_kv_write(cache(), **given)
    given.update(kw)
    with pytest.raises(ValueError):
        M.q1_kv_write(cache(), **given)
    assert len(library.calls) == 1


def test_read_gives_the_type_asked_for(library):
    c = cache(8, 128)
    slots = i32(1, 1, 20)
    k, v = M.q1_kv_read(c, slots)
    assert k.dtype == v.dtype == torch.bfloat16 and k.shape == (3, 2, 128)
    k, v = M.q1_kv_read(c, slots, torch.float32)
    assert k.dtype == torch.float32
    mine = z(3, 2, 128, dtype=torch.float16)
    k, v = M.q1_kv_read(c, slots, v=mine)
    assert v is mine and k.dtype == torch.float16
    with pytest.raises(ValueError):
        M.q1_kv_read(c, slots, torch.float32, v=mine)


def test_a_large_scratch_is_not_kept(monkeypatch):
    """A captured call, and one that needs much, has a workspace of its own; others share one."""
    made = []
    monkeypatch.setattr(D, "_empty", lambda n, dtype, device: made.append(n) or torch.empty(1, dtype=dtype).expand(n))
    monkeypatch.setattr(D, "_capturing", lambda: False)
    D._workspace(4096, 0, 99)
    D._workspace(4096, 0, 99)
    assert len(made) == 1
    for _ in range(2):
        D._workspace(D._KEEP + 1, 0, 99)
    assert len(made) == 3
    monkeypatch.setattr(D, "_capturing", lambda: True)
    D._workspace(4096, 0, 99)
    assert len(made) == 4
    D._scratch.kept.clear()
