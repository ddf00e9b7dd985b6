"""Attention over pages of 4 and 8 bits against the 64-bit oracle on the values the
pages hold: head layouts, types, page sizes, several queries a sequence, queries that
see nothing, garbage past the lengths, NaN in masked places and in what counts, ids
outside the pages, strided queries, streams, graph replays.  Tolerances are the
oracle's bounds plus the output's rounding."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as R
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


class Case:
    """Operands, and the values of each sequence's tokens; rows that are no token's hold garbage:
    NaN scales, codes that are NaN."""

    def __init__(self, seed, B, T, Hq, Hkv, D, lens, page, bits, dt, garbage=True, more=2):
        r = np.random.default_rng(seed)
        self.lens, self.page, self.bits, self.dt, self.T = lens, page, bits, dt, T
        per = max(1, -(-max(lens) // page))
        pages = B * per + more
        x = r.standard_normal((2, pages, Hkv, page, D)) * np.exp2(r.integers(-2, 3, (2, pages, Hkv, page, 1)))
        enc = [M.kv_encode(npd(torch.from_numpy(v).to(DT[dt])), bits, dt) for v in x]
        raw = [(M.pack(c, bits), s) for c, s in enc]
        self.table = r.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
        if garbage:
            used = np.zeros((pages, page), bool)
            for b, n in enumerate(lens):
                for i in range(n):
                    used[self.table[b, i // page], i % page] = True
            bad = np.broadcast_to(~used[:, None], (pages, Hkv, page))
            for c, s in raw:
                c[bad] = 0xff
                s[bad] = 0xff
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = Q.PackedKV(dev(raw[0][0]), dev(raw[1][0]), dev(raw[0][1]), dev(raw[1][1]), bits)
        self.q = torch.from_numpy(1.5 * r.standard_normal((B, T, Hq, D))).to(DT[dt]).cuda()
        self.table_dev, self.lens_dev = dev(self.table), torch.tensor(lens, dtype=torch.int32).cuda()

    def values(self, b):
        """(keys, values) [n, Hkv, D] of sequence b."""
        out = []
        for c, s in ((self.cache.k, self.cache.k_scales), (self.cache.v, self.cache.v_scales)):
            v = M.kv_decode(M.unpack(c.cpu().numpy(), self.bits), s.cpu().numpy(), self.bits)  # [pages, Hkv, page, D]
            v = v[self.table[b]].transpose(0, 2, 1, 3).reshape(-1, v.shape[1], v.shape[3])
            out.append(v[:self.lens[b]])
        return out

    def run(self, **kw):
        return Q.q1_kv_attn(self.q, self.cache, self.table_dev, self.lens_dev, **kw)

    def check(self, out, lse, out_dt, scale=None, what=""):
        D = self.q.shape[-1]
        scale = D ** -0.5 if scale is None else scale
        for b, n in enumerate(self.lens):
            keys, values = self.values(b)
            for t in range(self.T):
                m = max(0, n - (self.T - 1 - t))
                ref, bound, l, lb = R.prefix_attention(npd(self.q[b, t]), keys[:m], values[:m], scale)
                got, el = npd(out[b, t]), npd(lse[b, t])
                # values are 0 exactly here and there, and what is left may be below the normal numbers: a weight
                # and a product below 2^-126 each may be taken as 0, for m tokens m 2^-126 (1 + |v|)
                bound = bound + m * 2.0 ** -126 * (1 + np.abs(values[:m]).max(initial=0))
                over = np.abs(got - ref) - bound - R.half_ulp(np.abs(ref) + bound, out_dt)
                if t in (0, self.T - 1):
                    print(f"{what} sequence {b} query {t} of {m}: out over bound {over.max():.3g}", flush=True)
                assert np.isfinite(got).all() and over.max() <= 0, (b, t)
                if m == 0:
                    assert (el == -np.inf).all() and (got == 0).all()
                else:
                    assert (np.abs(el - l) <= lb).all(), (b, t)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,page,dt,out_dt", [
    (1, 1, 1, 1, 64, [1], 1, "bf16", "f32"),
    (1, 1, 8, 8, 128, [1], 16, "f16", "f32"),
    (4, 1, 24, 4, 128, [519, 0, 17, 128], 16, "bf16", "bf16"),
    (3, 1, 12, 2, 256, [300, 33, 64], 17, "bf16", "f32"),
    (5, 2, 8, 1, 64, [5, 300, 0, 129, 1], 48, "f16", "f16"),
    (2, 3, 6, 6, 128, [70, 257], 64, "bf16", "f32"),
    (3, 5, 8, 2, 128, [2, 700, 33], 16, "f16", "f32"),
    (9, 1, 6, 2, 64, [3 * i for i in range(9)], 1, "f16", "f32"),
    (2, 4, 32, 1, 256, [31, 94], 16, "bf16", "f32"),
    (2, 1, 40, 1, 64, [200, 3], 100, "bf16", "f32"),
    (1, 1, 4, 2, 128, [6000], 64, "bf16", "f32"),
    (1, 2, 4, 1, 256, [2500], 33, "f16", "f32"),
    (2, 60, 6, 2, 64, [61, 40], 16, "bf16", "f32"),
    (1, 150, 3, 1, 128, [150], 48, "f16", "f16"),
])
def test_against_oracle(B, T, Hq, Hkv, D, lens, page, dt, out_dt, bits):
    c = Case(B + T + D, B, T, Hq, Hkv, D, lens, page, bits, dt)
    out, lse = c.run(out_dtype=DT[out_dt])
    assert out.dtype == DT[out_dt]
    c.check(out, lse, out_dt, what=f"B={B} T={T} Hq={Hq}/{Hkv} D={D} {bits} bits")


@pytest.mark.parametrize("bits", [4, 8])
def test_nothing_to_see(bits):
    """Empty and negative lengths, no page in the table, no pages at all: zeros, lse = -infinity."""
    c = Case(2, 3, 2, 4, 2, 64, [0, 5, 1], 4, bits, "bf16")
    lens = torch.tensor([0, 5, -3], dtype=torch.int32).cuda()
    out, lse = Q.q1_kv_attn(c.q, c.cache, c.table_dev, lens)
    assert (out[[0, 2]] == 0).all() and (lse[[0, 2]] == -float("inf")).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()
    for cache, table in ((c.cache, c.table_dev[:, :0].contiguous()), (Q.PackedKV.empty(0, 4, 2, 64, bits), c.table_dev)):
        out, lse = Q.q1_kv_attn(c.q, cache, table, c.lens_dev)
        assert (out == 0).all() and (lse == -float("inf")).all()
    out, lse = Q.q1_kv_attn(c.q[:0], c.cache, c.table_dev[:0], c.lens_dev[:0])
    assert out.shape == (0, 2, 4, 64) and lse.shape == (0, 2, 4)
    out, lse = Q.q1_kv_attn(c.q[:, :0], c.cache, c.table_dev, c.lens_dev)
    assert out.shape == (3, 0, 4, 64)


def test_scores_far_apart():
    """Scores of thousands, equal and opposite: the maximum is taken out before exp."""
    c = Case(3, 2, 2, 4, 2, 64, [30, 150], 8, 4, "bf16")
    c.q = c.q * 100
    c.check(*c.run(out_dtype=torch.float32), "f32", what="large scores")
    c.check(*c.run(scale=0.0, out_dtype=torch.float32), "f32", scale=0.0, what="scale 0")
    c.check(*c.run(scale=-0.3, out_dtype=torch.float32), "f32", scale=-0.3, what="negative scale")


@pytest.mark.parametrize("bits", [4, 8])
def test_ids_and_lengths_out_of_range(bits):
    """A page id outside the pages leaves its tokens out; a length is clamped to the table."""
    c = Case(4, 2, 1, 4, 2, 128, [48, 48], 16, bits, "bf16", garbage=False)
    table = c.table.copy()
    table[0, 1], table[1, 2] = -7, 10 ** 6
    lens = torch.tensor([48, 10 ** 9], dtype=torch.int32).cuda()
    out, lse = Q.q1_kv_attn(c.q, c.cache, torch.from_numpy(table).cuda(), lens, out_dtype=torch.float32)
    for b, gone in ((0, range(16, 32)), (1, range(32, 48))):
        keep = [i for i in range(48) if i not in gone]
        keys, values = (x[keep] for x in c.values(b))
        ref, bound, l, lb = R.prefix_attention(npd(c.q[b, 0]), keys, values, 128 ** -0.5)
        assert (np.abs(npd(out[b, 0]) - ref) <= bound + R.half_ulp(ref, "f32")).all() and (np.abs(npd(lse[b, 0]) - l) <= lb).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,T,n", [(4, 2, 64, 3, 40), (6, 1, 128, 4, 200), (8, 2, 256, 2, 130), (12, 1, 128, 5, 6)])
def test_nan_blocks(Hq, Hkv, D, T, n, bits):
    """A NaN block of the last token: earlier queries do not see it.  Of a key: the row is NaN; of a value:
    its 32 columns."""
    for which in ("k", "v"):
        c = Case(T + n, 1, T, Hq, Hkv, D, [n], 16, bits, "bf16")
        scales = c.cache.k_scales if which == "k" else c.cache.v_scales
        want = [x.clone() for x in c.run(out_dtype=torch.float32)]
        page, at = c.table[0, (n - 1) // 16], (n - 1) % 16
        block = D // 32 - 1
        scales[page, Hkv - 1, at, block] = 255
        out, lse = c.run(out_dtype=torch.float32)
        last = slice((Hkv - 1) * (Hq // Hkv), Hq)
        assert torch.equal(out[:, :-1], want[0][:, :-1]) and torch.equal(lse[:, :-1], want[1][:, :-1])
        others = [h for h in range(Hq) if h < last.start]
        assert torch.equal(out[0, -1, others], want[0][0, -1, others])
        if which == "k":
            assert out[0, -1, last].isnan().all() and lse[0, -1, last].isnan().all()
        else:
            assert out[0, -1, last, 32 * block:].isnan().all() and torch.equal(lse, want[1])
            assert torch.equal(out[0, -1, last, :32 * block], want[0][0, -1, last, :32 * block])


def test_shared_pages_strided_queries_and_given_outputs():
    c = Case(5, 3, 2, 6, 2, 64, [40, 40, 40], 16, 4, "f16")
    c.table[1] = c.table[0]  # two sequences over the same pages
    c.table_dev = torch.from_numpy(c.table).cuda()
    a = c.run()
    big = torch.cat([torch.ones_like(c.q).flatten(2), c.q.flatten(2)], 2)
    q = big[..., 6 * 64:].unflatten(2, (6, 64))
    out, lse = torch.empty_like(c.q, dtype=torch.float32), torch.empty(3, 2, 6, device="cuda")
    b = Q.q1_kv_attn(q, c.cache, c.table_dev, c.lens_dev, out=out, lse=lse)
    assert b[0] is out and b[1] is lse and torch.equal(out.half(), a[0]) and torch.equal(lse, a[1])
    c.q[1] = c.q[0]
    out, lse = c.run()
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("T,lens", [(1, [40, 0, 2500, 1]), (3, [3000, 2, 129, 600])])
def test_graph_stream_and_bits(T, lens):
    c = Case(6, 4, T, 24, 4, 128, lens, 16, 4, "bf16")
    want = [x.clone() for x in c.run()]
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(c.run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.run()
    for i in range(4):
        got[0].zero_()
        got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        Q.q1_kv_attn(c.q * i, c.cache, c.table_dev, c.lens_dev)


def test_what_was_written_is_attended_to():
    """q1_kv_write, then attention, one token at a time and all at once."""
    r = np.random.default_rng(8)
    n, Hkv, D, page = 37, 2, 128, 16
    k, v = torch.from_numpy(r.standard_normal((2, n, Hkv, D))).bfloat16().cuda()
    q = torch.from_numpy(r.standard_normal((n, 6, D))).bfloat16().cuda()
    cache = Q.PackedKV.empty(4, page, Hkv, D)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32).cuda()
    slots = (table[0].repeat_interleave(page)[:n] * page + torch.arange(n, device="cuda") % page).to(torch.int32)
    steps = []
    for t in range(n):
        Q.q1_kv_write(cache, k[t:t + 1], v[t:t + 1], slots[t:t + 1])
        lens = torch.tensor([t + 1], dtype=torch.int32).cuda()
        steps.append(Q.q1_kv_attn(q[None, t:t + 1], cache, table, lens, out_dtype=torch.float32)[0][0, 0])
    whole = Q.q1_kv_attn(q[None], cache, table, torch.tensor([n], dtype=torch.int32).cuda(), out_dtype=torch.float32)[0][0]
    kk, vv = (npd(x) for x in Q.q1_kv_read(cache, slots))
    for t in range(n):
        ref, bound, _, _ = R.prefix_attention(npd(q[t]), kk[:t + 1], vv[:t + 1], D ** -0.5)
        for got in (steps[t], whole[t]):
            assert (np.abs(npd(got) - ref) <= bound + R.half_ulp(ref, "f32")).all()


@pytest.mark.parametrize("what", ["dtype", "table", "D", "host", "heads", "dims", "out"])
def test_binding_refusals(what):
    c = Case(7, 2, 1, 4, 2, 64, [3, 4], 4, 4, "bf16")
    q, table, lens, kw = c.q, c.table_dev, c.lens_dev, {}
    if what == "dtype":
        q = q.float()
    elif what == "table":
        table = table.long()
    elif what == "D":
        q = torch.cat([q, q], 3)
    elif what == "host":
        lens = lens.cpu()
    elif what == "heads":
        q = q[:, :, :3]
    elif what == "dims":
        q = q[:, 0]
    else:
        kw = dict(out=torch.empty(2, 1, 4, 32, device="cuda"))
    with pytest.raises((ValueError, Q.Q1Error)):
        Q.q1_kv_attn(q, c.cache, table, lens, **kw)


@pytest.mark.parametrize("bits", [4, 8])
def test_offsets_past_32_bits(bits):
    """A cache of over 4 GiB whose last pages are used."""
    c = Case(77, 2, 2, 8, 4, 128, [130, 65], 64, bits, "bf16")
    far = (5 << 30) // (64 * 4 * 128 * bits // 8)
    grow = lambda t: torch.cat([torch.zeros(far, *t.shape[1:], dtype=t.dtype, device="cuda"), t])  # noqa: E731
    big = Q.PackedKV(*(grow(t) for t in (c.cache.k, c.cache.v, c.cache.k_scales, c.cache.v_scales)), bits)
    want = c.run(out_dtype=torch.float32)
    got = Q.q1_kv_attn(c.q, big, c.table_dev + far, c.lens_dev, out_dtype=torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got, "f32", what="far")
