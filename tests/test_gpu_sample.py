"""The sampler on the GPU against the oracle: every filter alone and together,
ties, masked rows, infinities and NaN, one token to 152064 and beyond, types,
strided rows, graph replays.  The token has to be the one that the definition
gives, or, where the draw or a cut is that near to a boundary, one that it gives
for weights within 2^-22 of the oracle's: those are rounded from 64 bits, the
kernel's come from the 32-bit exponential (two units in the last place)."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as R

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


def dev(x, dt=torch.float32):
    return None if x is None else torch.tensor(x, dtype=dt).cuda()


def check(logits, u, T=None, k=None, p=None, m=None, what=""):
    tok, lp = Q.q1_sample(logits, dev(u), dev(T), dev(k, torch.int32), dev(p), dev(m))
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    host = logits.float().cpu().numpy()
    for b in range(len(u)):
        can = R.sample_choices(host[b], u[b], 1.0 if T is None else T[b], 0 if k is None else k[b],
                               1.0 if p is None else p[b], 0.0 if m is None else m[b])
        want = [l for t, l in can if t == tok[b]]
        assert want, f"{what} row {b}: token {tok[b]}, not {can[0][0]}"
        if tok[b] < 0:
            assert lp[b] == -np.inf
            continue
        # the token's weight and the sum are each within 2^-22, the logarithm within 2^-22 of itself;
        # a weight is floored by up to one unit of 2^-40 of the largest
        off = min(abs(lp[b] - l) - 2.0 ** -21 - 2.0 ** -22 * abs(l) - 1.0 / max(1.0, np.exp(l) * 2.0 ** 40) for l in want)
        assert off <= 0, f"{what} row {b}: logprob {lp[b]}, not {want[0]}"


def logits_of(seed, B, V, dt="f32", spread=2.0):
    r = np.random.default_rng(seed)
    x = spread * r.standard_normal((B, V))
    for b in range(B):
        x[b, r.integers(0, V, max(1, V // 50))] += 4.0
    return torch.from_numpy(x).to(DT[dt]).cuda()


@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 1000, 1025, 4097, 32003])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_filters(V, dt):
    r = np.random.default_rng(V)
    B = 12
    x = logits_of(V + 1, B, V, dt)
    u = r.uniform(0, 1, B).astype(np.float32).tolist()
    T = r.uniform(0.3, 2.0, B).astype(np.float32).tolist()
    k = r.integers(1, max(2, min(V, 300)), B).tolist()
    p = r.uniform(0.2, 0.99, B).astype(np.float32).tolist()
    m = r.uniform(0.001, 0.2, B).astype(np.float32).tolist()
    check(x, u, what="plain")
    check(x, u, T=T, what="temperature")
    check(x, u, T=T, k=k, what="top-k")
    check(x, u, T=T, p=p, what="top-p")
    check(x, u, T=T, m=m, what="min-p")
    check(x, u, T=T, k=k, p=p, m=m, what="all")
    check(x, u, T=[0.0] * B, k=k, p=p, m=m, what="greedy")


@pytest.mark.parametrize("B,V,dt", [(1, 152064, "f32"), (3, 152064, "bf16"), (70, 20011, "f16"), (2, 1 << 20, "f32")])
def test_large(B, V, dt):
    r = np.random.default_rng(B)
    x = logits_of(B, B, V, dt, spread=1.5)
    u = r.uniform(0, 1, B).astype(np.float32).tolist()
    check(x, u, p=[0.9] * B, k=[500] * B, what="large all")
    check(x, u, T=[0.7] * B, p=[0.95] * B, what="large top-p")
    check(x, u, T=[0.8] * B, what="large plain")


def test_ties():
    """Equal logits: the lowest index first, at the top-k and the top-p cut."""
    V, B = 5000, 9
    x = torch.zeros(B, V).cuda()
    x[:, 1000:1010] = 3.0
    x[:, 3:4000:7] = 1.0
    u = np.linspace(0.01, 0.99, B).astype(np.float32).tolist()
    for k in (1, 5, 10, 11, 300, 600, 4999):
        check(x, u, k=[k] * B, what=f"ties k={k}")
        check(x, u, k=[k] * B, p=[0.6] * B, what=f"ties k={k} p")
    for p in (0.001, 0.04, 0.3, 0.9):
        check(x, u, p=[p] * B, what=f"ties p={p}")
    check(torch.full((B, V), -7.5).cuda(), u, p=[0.5] * B, what="all equal")
    check(torch.zeros(B, V).cuda() * torch.tensor([1.0, -1.0]).cuda().repeat(V // 2), u, k=[3] * B, what="both zeros")


def test_masked_rows():
    """Rows with most or all logits at -infinity, at the type's lowest value or
    NaN; infinities."""
    inf, V, B = float("inf"), 700, 8
    base = logits_of(5, B, V)
    u = np.linspace(0.05, 0.95, B).astype(np.float32).tolist()
    x = base.clone()
    x[:, 10:] = -inf
    x[3] = -inf
    x[4, :] = float("nan")
    x[5, ::2] = float("nan")
    x[6, :] = torch.finfo(torch.float32).min
    check(x, u, what="masked")
    check(x, u, k=[50] * B, p=[0.9] * B, what="masked, filters")
    y = base.to(torch.bfloat16)
    y[:, 5:600] = torch.finfo(torch.bfloat16).min
    check(y, u, k=[300] * B, p=[0.97] * B, what="lowest value")
    z = base.clone()
    z[0, 7] = z[0, 500] = inf
    z[1, :] = inf
    z[2, 0], z[2, 1:] = 3e38, -3e38
    check(z, u, what="infinities")
    check(z, u, p=[0.7] * B, k=[2] * B, what="infinities, filters")


def test_parameters_at_their_edges():
    V, nan, inf = 300, float("nan"), float("inf")
    x = logits_of(6, 6, V)
    check(x, [0.0, 1.0, 2.0, -1.0, nan, 0.99999994], what="u")
    u = [0.3] * 6
    check(x, u, k=[0, -1, 1, V, V + 1, 2 ** 31 - 1], what="k")
    check(x, u, p=[0.0, -1.0, 1.0, 2.0, nan, 1e-30], what="p")
    check(x, u, m=[0.0, -1.0, 1.0, 2.0, nan, 1e-30], what="m")
    check(x, u, T=[0.0, -1.0, nan, 1e-30, inf, 1e4], what="T")


def test_strided_rows_and_types():
    x = logits_of(8, 5, 1003)
    wide = torch.full((5, 1500), 99.0).cuda()
    wide[:, :1003] = x
    u = dev([0.1, 0.3, 0.5, 0.7, 0.9])
    a = Q.q1_sample(wide[:, :1003], u, top_p=dev([0.9] * 5))
    b = Q.q1_sample(x, u, top_p=dev([0.9] * 5), tokens=torch.empty(5, dtype=torch.int32).cuda())
    assert b[0].dtype == torch.int32 and torch.equal(a[0], b[0].long()) and torch.equal(a[1], b[1])
    off = torch.empty(5 * 1003 + 1).cuda()[1:].view(5, 1003).copy_(x)  # 4-byte alignment only
    c = Q.q1_sample(off, u, top_p=dev([0.9] * 5))
    assert torch.equal(a[0], c[0])
    odd = torch.empty(5 * 1003 + 1, dtype=torch.bfloat16).cuda()[1:].view(5, 1003).copy_(x)
    d, e = Q.q1_sample(odd, u), Q.q1_sample(odd.clone(), u)
    assert torch.equal(d[0], e[0])


def test_batch_does_not_matter():
    """A row's token is the same alone, in a batch and on every call."""
    x = logits_of(9, 64, 152064, "bf16")
    u = torch.rand(64, generator=torch.Generator().manual_seed(1)).cuda()
    p = torch.full((64,), 0.9).cuda()
    t, lp = Q.q1_sample(x, u, top_p=p)
    t2, lp2 = Q.q1_sample(x, u, top_p=p)
    assert torch.equal(t, t2) and torch.equal(lp, lp2)
    for b in (0, 17, 63):
        t1, l1 = Q.q1_sample(x[b:b + 1], u[b:b + 1], top_p=p[b:b + 1])
        assert t1.item() == t[b].item() and l1.item() == lp[b].item()


def test_graph_and_stream():
    x = logits_of(10, 8, 30000)
    u = dev(np.linspace(0.03, 0.97, 8).astype(np.float32).tolist())
    k, p = dev([40] * 8, torch.int32), dev([0.9] * 8)
    want = [t.clone() for t in Q.q1_sample(x, u, top_k=k, top_p=p)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = Q.q1_sample(x, u, top_k=k, top_p=p)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = Q.q1_sample(x, u, top_k=k, top_p=p)
    for _ in range(4):
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        Q.q1_sample(x * 0.5, u, top_p=p)


@pytest.mark.parametrize("what", ["u", "k", "p", "host", "flat", "strided"])
def test_binding_refusals(what):
    x, u, k, p = logits_of(1, 2, 50), dev([0.1, 0.2]), None, None
    if what == "u":
        u = u.double()
    elif what == "k":
        k = torch.tensor([1, 2]).cuda()
    elif what == "p":
        p = dev([0.5])
    elif what == "host":
        u = u.cpu()
    elif what == "flat":
        x = x[0]
    else:
        x = x.t().contiguous().t()
    with pytest.raises(ValueError):
        Q.q1_sample(x, u, top_k=k, top_p=p)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_candidates(dt):
    """Cuts with few and with many candidates: top-k from one to more than half of
    the row, and top-p where the logits lie so near that a cut has hundreds beside it."""
    V = 30011
    k = [1, 2, 64, 255, 256, 257, 1000, 2047, 2048, 2049, 4096, 20000]
    B = len(k)
    u = np.linspace(0.02, 0.98, B).astype(np.float32).tolist()
    x = logits_of(11, B, V, dt)
    check(x, u, k=k, what="top-k")
    check(x, u, k=k, p=[0.9] * B, what="top-k and top-p")
    check(x, u, T=[1.3] * B, k=k, p=[0.5] * B, m=[0.01] * B, what="all")
    near = 0.05 * logits_of(12, B, V, dt)
    check(near, u, p=np.linspace(0.01, 0.99, B).astype(np.float32).tolist(), what="near, top-p")
    check(near, u, k=k, what="near, top-k")
    check(near, u, k=k, p=[0.7] * B, what="near, both")


def test_offsets_past_32_bits():
    """Rows so far apart that their offsets pass 32 bits."""
    B, V, ld = 5, 2000, 1 << 30
    x = logits_of(13, B, V, "bf16")
    wide = torch.empty((B - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((B, V), (ld, 1))
    wide.copy_(x)
    u = dev([0.1, 0.3, 0.5, 0.7, 0.9])
    for filters in (dict(), dict(top_p=dev([0.8] * B)), dict(top_k=dev([30] * B, torch.int32))):
        a, b = Q.q1_sample(wide, u, **filters), Q.q1_sample(x, u, **filters)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_weightless_logits_beside_the_cut():
    """A top-k cut among the smallest weights there are, with thousands of logits just below them that have
    none: these are no candidates.  The sum of what top-k keeps decides here whether top-p keeps token 0."""
    V, k, p = 20000, 400, np.float32(1 - 2.0 ** -24)
    r = np.random.default_rng(3)
    x = np.full(V, -100.0)
    at = 2 + r.permutation(V - 3)[:16000]
    x[at[:1000]] = -27.7245    # weight 1
    x[at[1000:]] = -27.732     # weight 0
    x[V - 1], x[1] = 0.0, -10.0
    # top-p keeps token 0 if token 1 and the largest lie below p times the sum: by 50 units here, less than
    # the units that top-k keeps
    others = 2.0 ** 40 + np.floor(np.exp(-10.0) * 2.0 ** 40)
    own = (others + 50) / float(p) - others - (k - 3)
    x[0] = np.log(own / 2.0 ** 40)
    row = torch.from_numpy(x).float().cuda()[None]
    assert R.sample(row[0].cpu().numpy(), 0.0, 1.0, k, float(p))[0] == 0
    check(row, [0.0], k=[k], p=[float(p)], what="weightless")


@pytest.mark.parametrize("V,dt", [(100, "f32"), (139, "bf16"), (201, "f16"), (454, "f32")])
def test_small_vocabularies(V, dt):
    """Large batches of short rows, every fourth with all filters, with top-k, with top-p and with none."""
    r = np.random.default_rng(V)
    B = 145
    x = logits_of(V + 5, B, V, dt)
    f = lambda lo, hi: r.uniform(lo, hi, B).astype(np.float32)  # noqa: E731
    row = np.arange(B) % 4
    k = np.where(row <= 1, r.integers(1, 200, B), 0).tolist()
    p = np.where(row % 2 == 0, f(0.7, 0.99), 1).astype(np.float32).tolist()
    m = np.where(row == 0, f(0, 0.1), 0).astype(np.float32).tolist()
    check(x, f(0, 1).tolist(), T=f(0.5, 1.3).tolist(), k=k, p=p, m=m, what="mixed")
