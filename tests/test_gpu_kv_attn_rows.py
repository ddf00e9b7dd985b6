"""Attention over quantised pages where many queries share each key/value head: whole
prompts over a table of many pages (the form by rows), items cut over workgroups and
not, lengths much shorter than the table, sequences with fewer tokens than queries,
NaN blocks and garbage, two captured graphs on one workspace.  Tolerances are those
of the small cases: the oracle's bounds plus the output's rounding."""
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
    yield
    torch.cuda.synchronize()


def npd(t):
    return t.detach().double().cpu().numpy()


class Prompts:
    """Sequences of `lens` tokens in tables for `capacity`, with every page behind the lengths
    an id outside the cache, and codes and scales of NaN in rows that are no token's."""

    def __init__(self, seed, B, T, Hq, Hkv, D, lens, page, bits, dt, capacity=4096):
        r = np.random.default_rng(seed)
        self.lens, self.page, self.bits, self.T, self.D = lens, page, bits, T, D
        per, wide = max(1, -(-max(lens) // page)), -(-capacity // page)
        pages = B * per + 1
        x = r.standard_normal((2, pages, Hkv, page, D)) * np.exp2(r.integers(-2, 3, (2, pages, Hkv, page, 1)))
        raw = [(M.pack(c, bits), s) for c, s in (M.kv_encode(npd(torch.from_numpy(v).to(DT[dt])), bits, dt) for v in x)]
        self.table = r.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            for i in range(n):
                used[self.table[b, i // page], i % page] = True
        for c, s in raw:
            c[np.broadcast_to(~used[:, None], (pages, Hkv, page))] = 0xff
            s[np.broadcast_to(~used[:, None], (pages, Hkv, page))] = 0xff
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = Q.PackedKV(dev(raw[0][0]), dev(raw[1][0]), dev(raw[0][1]), dev(raw[1][1]), bits)
        self.q = torch.from_numpy(1.5 * r.standard_normal((B, T, Hq, D))).to(DT[dt]).cuda()
        full = np.full((B, wide), pages + 5, np.int32)
        full[:, :per] = self.table
        self.table_dev, self.lens_dev = dev(full), torch.tensor(lens, dtype=torch.int32).cuda()

    def values(self, b):
        out = []
        for c, s in ((self.cache.k, self.cache.k_scales), (self.cache.v, self.cache.v_scales)):
            v = M.kv_decode(M.unpack(c.cpu().numpy(), self.bits), s.cpu().numpy(), self.bits)
            v = v[self.table[b]].transpose(0, 2, 1, 3).reshape(-1, v.shape[1], v.shape[3])
            out.append(v[:self.lens[b]])
        return out

    def run(self, **kw):
        return Q.q1_kv_attn(self.q, self.cache, self.table_dev, self.lens_dev, **kw)

    def check(self, out, lse, out_dt):
        out, lse, q = npd(out), npd(lse), npd(self.q)
        worst = -np.inf
        for b, n in enumerate(self.lens):
            keys, values = self.values(b)
            some = {0, 1, self.T // 2, self.T - 1, max(0, self.T - n - 1), min(self.T - 1, max(0, self.T - n)), *range(5, self.T, 41)}
            for t in sorted(some):
                m = max(0, n - (self.T - 1 - t))
                ref, bound, l, lb = R.prefix_attention(q[b, t], keys[:m], values[:m], self.D ** -0.5)
                bound = bound + m * 2.0 ** -126 * (1 + np.abs(values[:m]).max(initial=0))  # (products below the normal numbers)
                over = np.abs(out[b, t] - ref) - bound - R.half_ulp(np.abs(ref) + bound, out_dt)
                worst = max(worst, over.max())
                assert np.isfinite(out[b, t]).all() and over.max() <= 0, (b, t)
                if m == 0:
                    assert (lse[b, t] == -np.inf).all() and (out[b, t] == 0).all()
                else:
                    assert (np.abs(lse[b, t] - l) <= lb).all(), (b, t)
        print(f"out over bound {worst:.3g}", flush=True)


# rows of a key/value head: T * Hq / Hkv; items of 256 rows (128 of D 256), 128 of them or more
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,page,dt,out_dt", [
    (2, 512, 32, 16, 64, [512, 300], 16, "bf16", "f32"),
    (4, 512, 32, 16, 64, [100, 0, 513, 33], 64, "f16", "f16"),
    (4, 345, 24, 8, 128, [345, 600, 1, 64], 17, "bf16", "f32"),
    (1, 1030, 32, 8, 128, [1100], 128, "f16", "f32"),
    (1, 2100, 8, 8, 128, [63], 1, "bf16", "bf16"),
    (1, 700, 48, 8, 256, [700], 48, "bf16", "f32"),
    (2, 1024, 16, 8, 256, [65, 1300], 16, "f16", "f32"),
])
def test_prompts_against_oracle(B, T, Hq, Hkv, D, lens, page, dt, out_dt, bits):
    c = Prompts(B + T + D, B, T, Hq, Hkv, D, lens, page, bits, dt)
    out, lse = c.run(out_dtype=DT[out_dt])
    c.check(out, lse, out_dt)
    again = c.run(out_dtype=DT[out_dt])
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,Hkv", [(64, 32), (128, 32), (256, 16)])
def test_nan_blocks_reach_the_queries_that_see_them(D, Hkv, bits):
    """A NaN block of values is NaN in its 32 columns for the queries that see the token, and
    nowhere else; a NaN key makes the whole row NaN."""
    T, n, at = 1024, 1024, 777
    c = Prompts(D + bits, 1, T, Hkv, Hkv, D, [n], 64, bits, "bf16")
    clean, _ = c.run(out_dtype=torch.float32)
    page, row, blk = c.table[0, at // 64], at % 64, D // 32 - 1
    c.cache.v_scales[page, 3, row, blk] = 255
    out, lse = c.run(out_dtype=torch.float32)
    cols = slice(32 * blk, 32 * blk + 32)
    assert torch.isnan(out[0, at:, 3, cols]).all()
    other = out.clone()
    other[0, at:, 3, cols] = clean[0, at:, 3, cols]
    assert torch.equal(other, clean) and torch.isfinite(lse).all()
    c.cache.v_scales[page, 3, row, blk] = 127
    c.cache.k_scales[page, 5, row, 0] = 255
    out, lse = c.run(out_dtype=torch.float32)
    assert torch.isnan(out[0, at:, 5]).all() and torch.isfinite(out[0, :at]).all()
    assert torch.isfinite(out[0, :, [h for h in range(Hkv) if h not in (3, 5)]]).all()


def test_every_head_and_row_meets_its_own():
    """All heads and rows of a cut call against the same call one sequence at a time (other items)."""
    c = Prompts(11, 3, 700, 24, 8, 128, [700, 350, 900], 16, 8, "bf16")
    out, lse = c.run(out_dtype=torch.float32)
    for b in range(3):
        one, l1 = Q.q1_kv_attn(c.q[b:b + 1, 600:].contiguous(), c.cache, c.table_dev[b:b + 1].contiguous(), c.lens_dev[b:b + 1],
                               out_dtype=torch.float32)
        keys, values = c.values(b)
        # each is off by the weights' 2^-17 and fp32 sums, of values up to |v| and a softmax of 1: both forms within the oracle's
        # bound of one value, so apart by twice the largest bound
        _, bound, _, lb = R.prefix_attention(npd(c.q[b, 699]), keys, values, 128 ** -0.5)
        assert (out[b, 600:] - one[0]).abs().max().item() <= 4 * bound.max()
        assert torch.equal(torch.isinf(lse[b, 600:]), torch.isinf(l1[0]))


def test_two_graphs_share_a_stream():
    """Two captured calls of unlike shapes on one stream, replayed in turn with eager calls between."""
    a = Prompts(21, 2, 512, 32, 16, 64, [512, 300], 16, 4, "bf16")
    b = Prompts(22, 1, 700, 48, 8, 256, [700], 48, 8, "bf16")
    want = [x.run() for x in (a, b)]
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]
    graphs = []
    for x, o in zip((a, b), outs):
        x.run(out=o[0], lse=o[1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(out=o[0], lse=o[1])
        graphs.append(g)
    for turn in range(4):
        for g, o in zip(graphs, outs):
            for t in o:
                t.fill_(7.0)
            g.replay()
        a.run()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(w, o)), turn
