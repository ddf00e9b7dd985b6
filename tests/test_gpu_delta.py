"""The gated delta rule on the GPU against the 64-bit oracle: single tokens and
prompts, every head layout and type, ragged and empty sequences, slots outside
the pool, exact forgetting, strided operands, other streams, graph replays.
Tolerances are the oracle's error bounds plus the output's rounding."""
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


def draw(seed, lead, Hk, Hv, Dk, Dv, dt, l2, slots):
    """Operands as column slices of one projection's rows (so rows are strided)."""
    r = np.random.default_rng(seed)
    n = int(np.prod(lead))
    x = r.standard_normal((n, 2 * Hk * Dk + Hv * Dv + 8))
    if not l2:
        qk = x[:, :2 * Hk * Dk].reshape(n, 2 * Hk, Dk)
        x[:, :2 * Hk * Dk] = (qk / np.linalg.norm(qk, axis=-1, keepdims=True)).reshape(n, -1)
    x = torch.from_numpy(x).to(DT[dt]).cuda()
    cut = lambda a, h, d: x[:, a:a + h * d].view(n, h, d).view(*lead, h, d) if len(lead) == 1 else \
        x[:, a:a + h * d].unflatten(0, lead).unflatten(-1, (h, d))  # noqa: E731
    q, k, v = cut(0, Hk, Dk), cut(Hk * Dk, Hk, Dk), cut(2 * Hk * Dk, Hv, Dv)
    g = torch.from_numpy(-r.exponential(1.0, (*lead, Hv)) * r.choice([1e-3, 0.1, 2.0], Hv)).float().cuda()
    beta = torch.from_numpy(r.uniform(0, 1, (*lead, Hv))).float().cuda()
    state = torch.from_numpy(0.3 * r.standard_normal((slots, Hv, Dk, Dv))).float().cuda()
    return q, k, v, g, beta, state


def npd(t):
    return t.detach().double().cpu().numpy()


def check_sequence(q, k, v, g, beta, S0, l2, scale, c, out, S1, out_dt, what):
    ref, bound, S, sb = R.delta_rule(npd(q), npd(k), npd(v), npd(g), npd(beta), npd(S0), l2, scale, c)
    got, got_S = npd(out), npd(S1)
    eo = np.abs(got - ref) - bound - R.half_ulp(np.abs(ref) + bound, out_dt)
    es = np.abs(got_S - S) - sb
    print(f"{what}: worst out over bound {eo.max() if eo.size else 0:.3g}, state {es.max():.3g}", flush=True)
    assert not eo.size or (np.isfinite(got).all() and eo.max() <= 0), what
    assert np.isfinite(got_S).all() and es.max() <= 0, what


C_STEP = lambda Dk: 2 * Dk + 16              # noqa: E731
C_PREFILL = lambda Dk: 4 * (2 * Dk + 128) + 16  # noqa: E731


@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv,dt,out_dt,l2", [
    (1, 1, 16, 48, 128, 128, "bf16", "bf16", True),
    (8, 1, 4, 12, 128, 128, "bf16", "f32", True),
    (3, 4, 2, 2, 64, 64, "f16", "f16", False),
    (5, 1, 1, 6, 128, 64, "f16", "f32", True),
    (2, 2, 3, 3, 64, 16, "bf16", "f16", False),
    (33, 1, 1, 1, 64, 48, "bf16", "bf16", True),
    (2, 7, 2, 4, 128, 256, "f16", "bf16", True),
    (2, 3, 1, 2, 128, 208, "bf16", "f32", True),
])
def test_step(B, T, Hk, Hv, Dk, Dv, dt, out_dt, l2):
    q, k, v, g, beta, state = draw(B * 100 + T, (B, T), Hk, Hv, Dk, Dv, dt, l2, B + 3)
    slots = torch.from_numpy(np.random.default_rng(B).permutation(B + 3)[:B].astype(np.int32)).cuda()
    before = state.clone()
    out = Q.q1_delta_step(q, k, v, g, beta, state, slots, l2norm=l2, out_dtype=DT[out_dt])
    used = slots.tolist()
    for b in range(B):
        check_sequence(q[b], k[b], v[b], g[b], beta[b], before[used[b]], l2, Dk ** -0.5, C_STEP(Dk), out[b],
                       state[used[b]], out_dt, f"step sequence {b}")
    rest = [s for s in range(B + 3) if s not in used]
    assert torch.equal(state[rest], before[rest])


LENS = [1, 0, 63, 64, 65, 130, 7, 0, 200]


@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv,dt,out_dt,l2", [
    ([1], 16, 48, 128, 128, "bf16", "bf16", True),
    ([77], 2, 6, 128, 128, "bf16", "f32", True),
    (LENS, 2, 4, 128, 128, "f16", "f32", True),
    (LENS, 2, 2, 64, 64, "bf16", "bf16", False),
    (LENS, 1, 3, 64, 128, "f16", "f16", False),
    (LENS, 1, 2, 128, 48, "bf16", "f32", True),
    ([300, 20], 1, 1, 128, 256, "bf16", "f32", True),
    ([129], 1, 1, 64, 16, "f16", "f32", True),
    ([64, 64, 64], 1, 2, 128, 80, "f16", "f32", False),
    ([1100], 1, 2, 128, 128, "bf16", "f32", True),
])
def test_prefill(lens, Hk, Hv, Dk, Dv, dt, out_dt, l2):
    n, tokens = len(lens), sum(lens)
    q, k, v, g, beta, state = draw(tokens + Dv, (tokens,), Hk, Hv, Dk, Dv, dt, l2, n + 2)
    slots = torch.from_numpy(np.random.default_rng(n).permutation(n + 2)[:n].astype(np.int32)).cuda()
    cu = np.cumsum([0] + lens)
    before = state.clone()
    out = Q.q1_delta_prefill(q, k, v, g, beta, state, torch.from_numpy(cu.astype(np.int32)).cuda(), slots, l2norm=l2,
                             out_dtype=DT[out_dt])
    used = slots.tolist()
    for i in range(n):
        s = slice(int(cu[i]), int(cu[i + 1]))
        check_sequence(q[s], k[s], v[s], g[s], beta[s], before[used[i]], l2, Dk ** -0.5, C_PREFILL(Dk), out[s],
                       state[used[i]], out_dt, f"prefill sequence {i} of {lens[i]}")
        if lens[i] == 0:
            assert torch.equal(state[used[i]], before[used[i]])
    rest = [s for s in range(n + 2) if s not in used]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("kind", ["equal keys", "no decay", "fast decay", "no writes"])
def test_prefill_hard_chunks(kind):
    """Keys that repeat (the chunk's inverse is then as far from the identity as
    it gets), decays of zero and of hundreds a token, write strengths of one and zero."""
    T, Hk, Hv, D = 150, 1, 2, 128
    q, k, v, g, beta, state = draw(5, (T,), Hk, Hv, D, D, "bf16", True, 1)
    if kind == "equal keys":
        k = k[:1].expand(T, Hk, D).contiguous()
        beta.fill_(1.0)
        g.zero_()
    elif kind == "no decay":
        g.zero_()
        beta.fill_(1.0)
    elif kind == "fast decay":
        g.copy_(-300 * torch.rand_like(g))
    else:
        beta.zero_()
    before = state.clone()
    out = Q.q1_delta_prefill(q, k, v, g, beta, state, torch.tensor([0, T], dtype=torch.int32).cuda(), l2norm=True,
                             out_dtype=torch.float32)
    # the inverse of a chunk of equal keys has row sums of up to 2; it is made
    # from rows of ones, whose products have up to 64 terms of size one
    check_sequence(q, k, v, g, beta, before[0], True, D ** -0.5, 4 * C_PREFILL(D), out, state[0], "f32", kind)


@pytest.mark.parametrize("prefill", [False, True])
def test_forget_exactly(prefill):
    """g = -infinity drops the state whatever it holds (large values, not NaN)."""
    T, D = 100, 128
    q, k, v, g, beta, state = draw(9, (T,), 1, 2, D, D, "bf16", True, 1)
    g[70] = -float("inf")
    g[3, 1] = -float("inf")
    state *= 1e3
    before = state.clone()
    if prefill:
        out = Q.q1_delta_prefill(q, k, v, g, beta, state, torch.tensor([0, T], dtype=torch.int32).cuda(), l2norm=True,
                                 out_dtype=torch.float32)
    else:
        out = Q.q1_delta_step(q[None], k[None], v[None], g[None], beta[None], state, l2norm=True,
                              out_dtype=torch.float32)[0]
    check_sequence(q, k, v, g, beta, before[0], True, D ** -0.5, C_PREFILL(D) if prefill else C_STEP(D), out, state[0],
                   "f32", "forget")


@pytest.mark.parametrize("prefill", [False, True])
def test_slots_outside_the_pool(prefill):
    B, T, D = 4, 3, 64
    q, k, v, g, beta, state = draw(3, (B, T), 1, 2, D, D, "bf16", True, 4)
    before = state.clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32).cuda()
    if prefill:
        flat = [x.flatten(0, 1) for x in (q, k, v, g, beta)]
        out = Q.q1_delta_prefill(*flat, state, torch.arange(0, 13, 3, dtype=torch.int32).cuda(), slots, l2norm=True)
        out = out.view(B, T, 2, D)
    else:
        out = Q.q1_delta_step(q, k, v, g, beta, state, slots, l2norm=True)
    assert (out[1:3] == 0).all() and (out[0] != 0).any() and (out[3] != 0).any()
    assert torch.equal(state[[1, 3]], before[[1, 3]])
    assert not torch.equal(state[2], before[2]) and not torch.equal(state[0], before[0])


def test_offsets_are_clamped():
    """Offsets outside [0, tokens] read and write nothing outside the rows."""
    T, D = 90, 64
    q, k, v, g, beta, state = draw(4, (T,), 1, 1, D, D, "bf16", True, 2)
    s2 = state.clone()
    a = Q.q1_delta_prefill(q, k, v, g, beta, state, torch.tensor([-5, 40, 4000], dtype=torch.int32).cuda(), l2norm=True)
    b = Q.q1_delta_prefill(q, k, v, g, beta, s2, torch.tensor([0, 40, T], dtype=torch.int32).cuda(), l2norm=True)
    assert torch.equal(a, b) and torch.equal(state, s2)


def test_rows_past_a_sequence_do_not_matter():
    """NaN in rows that belong to no sequence, and in the next one, stay there."""
    T, D = 100, 128
    q, k, v, g, beta, state = draw(6, (T,), 1, 2, D, D, "bf16", True, 2)
    s2 = state.clone()
    cu = torch.tensor([0, 70, 70], dtype=torch.int32).cuda()
    a = Q.q1_delta_prefill(q, k, v, g, beta, state, cu, l2norm=True)
    q, k, v = (x.clone() for x in (q, k, v))
    for x in (q, k, v, g, beta):
        x[70:] = float("nan")
    b = Q.q1_delta_prefill(q, k, v, g, beta, s2, cu, l2norm=True)
    assert torch.equal(a[:70], b[:70]) and torch.equal(state, s2) and torch.isfinite(s2).all()


def test_same_bits_every_time():
    q, k, v, g, beta, state = draw(7, (333,), 2, 4, 128, 128, "bf16", True, 2)
    cu = torch.tensor([0, 100, 333], dtype=torch.int32).cuda()
    first = None
    for _ in range(3):
        s = state.clone()
        o = Q.q1_delta_prefill(q, k, v, g, beta, s, cu, l2norm=True)
        if first is None:
            first = (o, s)
        assert torch.equal(o, first[0]) and torch.equal(s, first[1])


def test_graph_and_other_stream():
    q, k, v, g, beta, state = draw(8, (150,), 2, 4, 128, 128, "bf16", True, 2)
    cu = torch.tensor([0, 60, 150], dtype=torch.int32).cuda()
    sq, sk, sv = (x[:2].view(2, 1, *x.shape[1:]) for x in (q.contiguous(), k.contiguous(), v.contiguous()))
    sg, sb = g[:2].view(2, 1, -1).contiguous(), beta[:2].view(2, 1, -1).contiguous()
    start = state.clone()

    def go(st):
        st.copy_(start)
        a = Q.q1_delta_prefill(q, k, v, g, beta, st, cu, l2norm=True)
        return a, Q.q1_delta_step(sq, sk, sv, sg, sb, st, l2norm=True)

    want = [x.clone() for x in go(state)] + [state.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = go(state)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip((*got, state), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go(state)
    for _ in range(4):
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*got, state), want))
        (want[0].float().sum() + 1).item()


def test_step_continues_prefill():
    """A prompt in two calls and a token after it equal one longer prompt, to
    the bound of the two."""
    T, D = 131, 128
    q, k, v, g, beta, state = draw(11, (T,), 1, 2, D, D, "bf16", True, 1)
    start = state.clone()
    Q.q1_delta_prefill(q[:70], k[:70], v[:70], g[:70], beta[:70], state, torch.tensor([0, 70], dtype=torch.int32).cuda(), l2norm=True)
    Q.q1_delta_prefill(q[70:130], k[70:130], v[70:130], g[70:130], beta[70:130], state,
                       torch.tensor([0, 60], dtype=torch.int32).cuda(), l2norm=True)
    out = Q.q1_delta_step(q[130:][None], k[130:][None], v[130:][None], g[130:][None], beta[130:][None], state,
                          l2norm=True, out_dtype=torch.float32)
    ref, bound, S, sb = R.delta_rule(npd(q), npd(k), npd(v), npd(g), npd(beta), npd(start[0]), True, D ** -0.5, C_PREFILL(D))
    assert (np.abs(npd(out)[0, 0] - ref[-1]) <= bound[-1] + R.half_ulp(ref[-1], "f32")).all()
    assert (np.abs(npd(state[0]) - S) <= sb).all()


@pytest.mark.parametrize("what", ["shape", "dtype", "state", "strided", "host", "slots"])
def test_binding_refusals(what):
    q, k, v, g, beta, state = draw(1, (2, 1), 2, 2, 64, 64, "bf16", True, 2)
    slots = None
    if what == "shape":
        k = k[:1]
    elif what == "dtype":
        v = v.half()
    elif what == "state":
        state = state.double()
    elif what == "strided":
        q = q.transpose(-1, -2).contiguous().transpose(-1, -2)
    elif what == "host":
        g = g.cpu()
    else:
        slots = torch.zeros(3, dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        Q.q1_delta_step(q, k, v, g, beta, state, slots, l2norm=True)


def test_offsets_past_32_bits():
    """States at the end of a pool of over 4 GiB, and tokens so far apart that their
    offsets pass 32 bits: the same results as for small operands."""
    Hk, Hv, D, T, ld = 1, 2, 128, 9000, 1 << 18
    q, k, v, g, beta, state = draw(9, (T,), Hk, Hv, D, D, "bf16", True, 3)
    slots = 40000
    pool = torch.empty(slots, Hv, D, D, device="cuda")
    pool[-3:] = state
    cu = torch.tensor([0, 5, T], dtype=torch.int32).cuda()
    at = torch.tensor([2, 0], dtype=torch.int32).cuda()
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, 4 * D), (ld, 1))
    wide[:, :D], wide[:, D:2 * D], wide[:, 2 * D:] = q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)
    far = lambda a, h: wide[:, a:a + h * D].unflatten(1, (h, D))  # noqa: E731
    for step in (False, True):
        if step:
            n = 2
            args = [x.reshape(2, T // 2, *x.shape[1:]) if x.is_contiguous() else x.unflatten(0, (2, T // 2))
                    for x in (q, k, v, g, beta)]
            wargs = [x.unflatten(0, (2, T // 2)) for x in (far(0, Hk), far(D, Hk), far(2 * D, Hv))]
            want = Q.q1_delta_step(*args, state, at[:n], l2norm=True)
            got = Q.q1_delta_step(*wargs, *args[3:], pool, at[:n] + (slots - 3), l2norm=True)
        else:
            want = Q.q1_delta_prefill(q, k, v, g, beta, state, cu, at, l2norm=True)
            got = Q.q1_delta_prefill(far(0, Hk), far(D, Hk), far(2 * D, Hv), g, beta, pool, cu, at + (slots - 3), l2norm=True)
        assert torch.equal(got, want) and torch.equal(pool[-3:], state)


@pytest.mark.parametrize("nseq,Hk,Hv", [(64, 1, 3), (65, 2, 8), (150, 1, 1)])
def test_many_sequences(nseq, Hk, Hv):
    """Batches of many short sequences, empty ones among them: every one is done, whatever
    the order they are started in."""
    r = np.random.default_rng(nseq)
    lens = r.integers(0, 90, nseq) * (r.random(nseq) < 0.8)
    cu, D = np.cumsum([0, *lens]), 64
    q, k, v, g, beta, state = draw(nseq, (int(cu[-1]),), Hk, Hv, D, D, "bf16", True, nseq)
    slots = torch.from_numpy(r.permutation(nseq).astype(np.int32)).cuda()
    before = state.clone()
    out = Q.q1_delta_prefill(q, k, v, g, beta, state, torch.from_numpy(cu.astype(np.int32)).cuda(), slots, l2norm=True,
                             out_dtype=torch.float32)
    for i, s in enumerate(slots.tolist()):
        at = slice(int(cu[i]), int(cu[i + 1]))
        check_sequence(q[at], k[at], v[at], g[at], beta[at], before[s], True, D ** -0.5, C_PREFILL(D), out[at], state[s],
                       "f32", f"sequence {i} of {lens[i]}")
