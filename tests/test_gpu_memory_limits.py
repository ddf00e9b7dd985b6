"""Calls at the edges of what decoder memory allows: more sequences than a workgroup
has lanes, more parts of a row than a wave, threads on one stream, captured calls
that are replayed on several streams at once, a first call under capture."""
import threading

import numpy as np
import pytest
import torch

from oracle import decode_oracle as R
from oracle import memory_oracle as M

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    yield
    torch.cuda.synchronize()


def npd(t):
    return t.detach().double().cpu().numpy()


def pages_of(seed, B, Hkv, D, lens, page, bits, wide):
    """Random pages, one after the other for each sequence; the table has room for `wide`."""
    r = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    pages = max(1, sum(per))
    x = r.standard_normal((2, pages, Hkv, page, D)).astype(np.float32)
    cache = Q.PackedKV.empty(pages, page, Hkv, D, bits)
    slots = torch.arange(pages * page, dtype=torch.int32).cuda()
    rows = [torch.from_numpy(v).bfloat16().cuda().transpose(1, 2).reshape(-1, Hkv, D) for v in x]
    Q.q1_kv_write(cache, rows[0], rows[1], slots)
    table = np.zeros((B, wide), np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = np.arange(at, at + n)
        at += n
    k, v = (npd(t) for t in Q.q1_kv_read(cache, slots, torch.float32))
    values = []
    at = 0
    for n, m in zip(lens, per):
        values.append((k[at:at + n], v[at:at + n]))
        at += m * page
    return cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), values


def check(q, out, lse, values, T=1):
    D = q.shape[-1]
    for b, (k, v) in enumerate(values):
        for t in range(T):
            m = max(0, len(k) - (T - 1 - t))
            ref, bound, l, lb = R.prefix_attention(npd(q[b, t]), k[:m], v[:m], D ** -0.5)
            bound = bound + m * 2.0 ** -126 * (1 + np.abs(v[:m]).max(initial=0))  # (products below the normal numbers)
            assert (np.abs(npd(out[b, t]) - ref) <= bound + R.half_ulp(np.abs(ref) + bound, "f32")).all(), (b, t)
            assert (np.abs(npd(lse[b, t]) - l) <= lb).all() if m else (npd(lse[b, t]) == -np.inf).all(), (b, t)


@pytest.mark.parametrize("B,Hq,Hkv,D,T", [(300, 2, 1, 64, 1), (700, 1, 1, 128, 1), (140, 4, 2, 64, 2)])
def test_many_sequences_of_unlike_lengths(B, Hq, Hkv, D, T):
    r = np.random.default_rng(B)
    lens = [int(n) for n in r.integers(0, 90, B)]
    lens[B // 3], lens[-1], lens[0] = 9000, 700, 0
    cache, table, n, values = pages_of(B, B, Hkv, D, lens, 64, 4, 160)
    q = torch.from_numpy(r.standard_normal((B, T, Hq, D))).bfloat16().cuda()
    out, lse = Q.q1_kv_attn(q, cache, table, n, out_dtype=torch.float32)
    check(q, out, lse, values, T)


@pytest.mark.parametrize("T,group,D", [(1, 1, 64), (2, 12, 128), (1, 3, 256)])
def test_a_row_of_very_many_parts(T, group, D):
    """Two sequences of which one has nearly all units: over a hundred workgroups share its item."""
    lens = [40000, 1]
    cache, table, n, values = pages_of(7, 2, 1, D, lens, 128, 8, 320)
    q = torch.from_numpy(np.random.default_rng(8).standard_normal((2, T, group, D))).bfloat16().cuda()
    out, lse = Q.q1_kv_attn(q, cache, table, n, out_dtype=torch.float32)
    check(q, out, lse, values, T)


def calls(seed):
    """One call of each kind that has a workspace: a function that makes them, on tensors of its own."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    lens = [5000, 300 + seed]
    cache, table, n, _ = pages_of(seed, 2, 2, 64, lens, 32, 4, 160)
    q = r(2, 1, 8, 64).bfloat16()
    Di, N, T = 64, 16, 700
    x, dt, z, Bm, Cm = (r(T, w).bfloat16() for w in (Di, Di, Di, N, N))
    A, D = -r(Di, N).exp(), r(Di)
    cu = torch.tensor([0, 500, T], dtype=torch.int32).cuda()
    taps, rows0, h0 = r(Di, 4).bfloat16(), r(2, 3, Di).bfloat16(), r(2, Di, N)

    def run():
        out, lse = Q.q1_kv_attn(q, cache, table, n)
        h, rows = h0.clone(), rows0.clone()
        mixed = Q.q1_conv_prefill(x, taps, rows, cu)
        y = Q.q1_scan_prefill(mixed, dt, A, Bm, Cm, h, cu, D=D, z=z)
        return out, lse, rows, y, h

    return run


def test_threads_on_one_stream():
    runs = [calls(i) for i in range(3)]
    want = [[t.clone() for t in run()] for run in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]

    def work(i):
        for _ in range(25):
            got[i].append(runs[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert len(got[i]) == 25
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, w))


def test_captured_calls_on_two_streams_at_once():
    """Each captured call has a workspace of its own: two of them may be replayed at the same
    time, with eager calls beside them."""
    runs = [calls(10), calls(11)]
    want = [[t.clone() for t in run()] for run in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for run in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(6):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        eager = runs[0]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
            for t in o:
                t.zero_()
        torch.cuda.synchronize()


def test_a_captured_call_that_no_eager_one_came_before():
    """Shapes and types that nothing above has run."""
    r = torch.Generator().manual_seed(3)
    q = torch.randn(3, 1, 2, 256, generator=r).half().cuda()
    cache, table, n, values = pages_of(3, 3, 2, 256, [5000, 0, 77], 16, 8, 400)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = Q.q1_kv_attn(q, cache, table, n, out_dtype=torch.float32)
    for _ in range(3):
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check(q, out, lse, values)


def test_the_same_page_many_times():
    """A table may name a page as often as it likes, for several sequences."""
    cache, _, _, values = pages_of(4, 1, 2, 64, [48], 16, 4, 3)
    order = [[2, 2, 0, 2, 1], [1, 1, 1, 1, 1]]
    k, v = values[0]
    pick = [np.concatenate([np.arange(16 * p, 16 * p + 16) for p in o]) for o in order]
    lens = [80, 67]
    q = torch.randn(2, 3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out, lse = Q.q1_kv_attn(q, cache, torch.tensor(order, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            out_dtype=torch.float32)
    check(q, out, lse, [(k[p][:m], v[p][:m]) for p, m in zip(pick, lens)], 3)


@pytest.mark.parametrize("bits", [4, 8])
def test_masks_of_the_types_extremes(bits):
    """Keys of the largest values and queries of the largest of their type: scores of infinity make
    the row NaN where they are seen, and nothing where they are not; scores of -infinity weigh nothing."""
    cache = Q.PackedKV.empty(2, 4, 1, 64, bits)
    k = torch.zeros(8, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.arange(8, device="cuda", dtype=torch.bfloat16)[:, None, None].expand(8, 1, 64).contiguous()
    k[3] = -3e38  # score -infinity
    k[6] = 3e38   # score +infinity
    Q.q1_kv_write(cache, k, v, torch.arange(8, dtype=torch.int32, device="cuda"))
    q = torch.full((1, 1, 1, 64), 1e30, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    held = Q.q1_kv_read(cache, torch.arange(8, dtype=torch.int32, device="cuda"), torch.float32)[1][:, 0, 0]
    for n, seen in ((3, [0, 1, 2]), (4, [0, 1, 2]), (6, [0, 1, 2, 4, 5])):
        out, lse = Q.q1_kv_attn(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
        want = held[seen].mean().item()  # scores 0
        # weights 1 and sums of them exact; one division, one product, rounded each
        assert (out - want).abs().max().item() <= 2 * 2.0 ** -24 * want + 1e-30
        assert abs(lse.item() - np.log(len(seen))) <= 4e-7
    out, lse = Q.q1_kv_attn(q, cache, table, torch.tensor([8], dtype=torch.int32, device="cuda"))
    assert torch.isnan(out).all()
