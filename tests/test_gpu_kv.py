"""Keys and values quantised into pages and read back: bit for bit the oracle's codes,
scales and values; every type and head layout, ties, zeros, subnormals, the ends of
the scales, NaN and infinities, slots outside the pages, strided rows, other streams,
graph replays."""
import numpy as np
import pytest
import torch

from oracle import memory_oracle as M

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield
    torch.cuda.synchronize()


def npd(t):
    return t.detach().double().cpu().numpy()


def rows_of(cache, slots):
    """(k codes, k scales, v codes, v scales) of the slots' rows, [rows, Hkv, ..]."""
    at = slots.long().cpu().numpy()
    page, off = at // cache.page_size, at % cache.page_size
    return [t.cpu().numpy()[page, :, off] for t in (cache.k, cache.k_scales, cache.v, cache.v_scales)]


def fill(cache, byte=0x5b):
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        t.fill_(byte)


def check(cache, k, v, slots, dt):
    got = rows_of(cache, slots)
    for x, codes, scales in ((k, *got[:2]), (v, *got[2:])):
        c, s = M.kv_encode(npd(x), cache.bits, dt)
        assert (scales == s).all()
        assert (codes == M.pack(c, cache.bits)).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,Hkv,D,page,dt", [
    (1, 1, 64, 1, "bf16"), (3, 2, 128, 16, "f16"), (40, 4, 256, 17, "bf16"), (130, 3, 64, 48, "f16"), (257, 8, 128, 64, "bf16"),
])
def test_against_oracle(tokens, Hkv, D, page, dt, bits):
    r = np.random.default_rng(tokens + D + bits)
    x = r.standard_normal((2, tokens, Hkv, D)) * np.exp2(r.integers(-12, 6, (2, tokens, Hkv, 1)))
    x[:, :, :, ::7] *= 9
    k, v = torch.from_numpy(x).to(DT[dt]).cuda()
    pages = -(-tokens // page) + 2
    cache = Q.PackedKV.empty(pages, page, Hkv, D, bits)
    fill(cache)
    slots = torch.from_numpy(r.permutation(pages * page)[:tokens].astype(np.int32)).cuda()
    Q.q1_kv_write(cache, k, v, slots)
    check(cache, k, v, slots, dt)
    left = torch.ones(pages * page, dtype=torch.bool)
    left[slots.long().cpu()] = False
    for t in rows_of(cache, left.nonzero()[:, 0]):
        assert (t == 0x5b).all()  # no other row is touched
    for out_dt in ("bf16", "f16", "f32"):
        back = Q.q1_kv_read(cache, slots, out_dtype=DT[out_dt])
        for x, got in zip((k, v), back):
            want = torch.from_numpy(M.kv_decode(*M.kv_encode(npd(x), bits, dt), bits)).to(DT[out_dt])
            assert got.dtype == DT[out_dt] and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_pattern_of_the_type(bits, dt):
    """All 65536 patterns, as the largest of a block and beside a larger one: ties, subnormals, the ends of
    the scales, NaN and infinities."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dt])
    x = torch.zeros(2, 1024, 64, 32, dtype=DT[dt])
    x[0].view(65536, 32)[:, 5] = every
    x[0].view(65536, 32)[:, 31] = 0.3 * every
    # a block whose scale comes from its first element, the others all patterns below it
    x[1].view(65536, 32)[:] = every.view(2048, 32).repeat(32, 1)
    finite = torch.isfinite(x[1].view(32, 2048, 32))
    for i in range(32):
        x[1].view(32, 2048, 32)[i] = torch.where(finite[i], x[1].view(32, 2048, 32)[i], torch.zeros((), dtype=DT[dt]))
        x[1].view(32, 2048, 32)[i, :, 0] = 2.0 ** (i - 15) * (1 + (i % 4) / 4)
    x = x.view(2, 1024, 16, 128).cuda()
    cache = Q.PackedKV.empty(1, 1024, 16, 128, bits)
    slots = torch.arange(1024, dtype=torch.int32).cuda()
    Q.q1_kv_write(cache, x[0], x[1], slots)
    check(cache, x[0], x[1], slots, dt)
    for got, src in zip(Q.q1_kv_read(cache, slots, out_dtype=torch.float32), x):
        want = M.kv_decode(*M.kv_encode(npd(src), bits, dt), bits)
        assert np.array_equal(npd(got), want, equal_nan=True)


@pytest.mark.parametrize("bits", [4, 8])
def test_slots_outside_and_repeated_reads(bits):
    r = np.random.default_rng(5)
    k, v = torch.from_numpy(r.standard_normal((2, 6, 2, 64))).bfloat16().cuda()
    cache = Q.PackedKV.empty(3, 4, 2, 64, bits)
    fill(cache, 0x22)
    slots = torch.tensor([3, -1, 12, 11, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    Q.q1_kv_write(cache, k, v, slots)
    inside = slots[[0, 3]]
    check(cache, k[[0, 3]], v[[0, 3]], inside, "bf16")
    others = torch.tensor([s for s in range(12) if s not in (3, 11)])
    assert all((t == 0x22).all() for t in rows_of(cache, others))
    gk, gv = Q.q1_kv_read(cache, torch.tensor([11, 12, 3, 11, -5], dtype=torch.int32).cuda())
    assert gk.dtype == torch.bfloat16 and not gk[[1, 4]].any() and not gv[[1, 4]].any()
    assert torch.equal(gk[0], gk[3]) and torch.equal(gv[0], gv[3]) and gk[0].any()
    want = torch.from_numpy(M.kv_decode(*M.kv_encode(npd(k[0]), bits, "bf16"), bits)).bfloat16()
    assert torch.equal(gk[2].cpu(), want)


def test_no_pages_and_no_rows():
    cache = Q.PackedKV.empty(0, 16, 2, 64)
    x = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.arange(3, dtype=torch.int32).cuda()
    Q.q1_kv_write(cache, x, x, slots)
    k, v = Q.q1_kv_read(cache, slots)
    assert not k.any() and not v.any()
    cache = Q.PackedKV.empty(1, 16, 2, 64)
    Q.q1_kv_write(cache, x[:0], x[:0], slots[:0])
    assert Q.q1_kv_read(cache, slots[:0])[0].shape == (0, 2, 64) and not cache.k.any()


def test_strided_rows_given_outputs_streams_and_graphs():
    r = np.random.default_rng(9)
    tokens, Hkv, D = 77, 2, 128
    x = torch.from_numpy(r.standard_normal((tokens, 8 + 2 * Hkv * D))).half().cuda()
    k, v = (x[:, 8 + i * Hkv * D:8 + (i + 1) * Hkv * D].unflatten(1, (Hkv, D)) for i in range(2))
    slots = torch.from_numpy(r.permutation(96)[:tokens].astype(np.int32)).cuda()
    plain, other = Q.PackedKV.empty(6, 16, Hkv, D), Q.PackedKV.empty(6, 16, Hkv, D)
    Q.q1_kv_write(plain, k.contiguous(), v.contiguous(), slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.q1_kv_write(other, k, v, slots)
        got = Q.q1_kv_read(other, slots)
    torch.cuda.current_stream().wait_stream(side)
    want = Q.q1_kv_read(plain, slots)
    assert torch.equal(plain.k, other.k) and torch.equal(plain.v_scales, other.v_scales)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    given = torch.empty(tokens, Hkv, D, device="cuda"), torch.empty(tokens, Hkv, D, device="cuda")
    back = Q.q1_kv_read(plain, slots, k=given[0], v=given[1])
    assert back[0] is given[0] and torch.equal(given[1].bfloat16(), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.q1_kv_write(other, k, v, slots)
        got = Q.q1_kv_read(other, slots)
    for i in range(3):
        x.normal_()
        graph.replay()
        Q.q1_kv_write(plain, k, v, slots)
        want = Q.q1_kv_read(plain, slots)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(plain.k, other.k)


def test_offsets_past_32_bits():
    """Pages of over 4 GiB: the last ones are written and read as the first ones are."""
    page, Hkv, D = 64, 8, 128
    pages = (5 << 30) // (page * Hkv * D // 2)
    cache = Q.PackedKV.empty(pages, page, Hkv, D)
    r = np.random.default_rng(3)
    k, v = torch.from_numpy(r.standard_normal((2, 5, Hkv, D))).bfloat16().cuda()
    far = torch.arange(pages * page - 5, pages * page, dtype=torch.int32).cuda()
    Q.q1_kv_write(cache, k, v, far)
    small = Q.PackedKV.empty(1, page, Hkv, D)
    near = torch.arange(5, dtype=torch.int32).cuda()
    Q.q1_kv_write(small, k, v, near)
    assert all(torch.equal(a, b) for a, b in zip(Q.q1_kv_read(cache, far), Q.q1_kv_read(small, near)))
    assert not Q.q1_kv_read(cache, near)[0].any()


@pytest.mark.parametrize("what", ["dtype", "heads", "slots", "host", "mixed", "inner"])
def test_binding_refusals(what):
    cache = Q.PackedKV.empty(2, 4, 2, 64)
    k = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    v, slots = k.clone(), torch.arange(3, dtype=torch.int32).cuda()
    if what == "dtype":
        k, v = k.float(), v.float()
    elif what == "heads":
        k = k[:, :1]
    elif what == "slots":
        slots = slots.long()
    elif what == "host":
        slots = slots.cpu()
    elif what == "mixed":
        v = v.half()
    else:
        k = torch.zeros(3, 64, 2, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    with pytest.raises((ValueError, Q.Q1Error)):
        Q.q1_kv_write(cache, k, v, slots)
