"""The selective state space scan on the GPU against the 64-bit oracle: single tokens and
prompts, state sizes and types, ragged and empty sequences, with and without gate, skip
and bias, slots outside the pool, rows of no sequence, strided operands, decays of 0 and
1, NaN and infinities, streams, graph replays."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as R
from oracle import memory_oracle as M

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PIECE = 512  # tokens a piece of these prompts has at most


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield
    torch.cuda.synchronize()


def npd(t):
    return None if t is None else t.detach().double().cpu().numpy()


def draw(seed, lead, Di, N, dt, dt32, slots, full=True):
    """Operands as column slices of one projection's rows."""
    r = np.random.default_rng(seed)
    rows = int(np.prod(lead))
    dev = lambda a, t: torch.from_numpy(a).to(DT[t]).cuda()  # noqa: E731
    x = dev(r.standard_normal((rows, 2 * Di + 2 * N + 16)), dt)
    cut = lambda a, n: x[:, a:a + n].unflatten(0, lead) if len(lead) > 1 else x[:, a:a + n]  # noqa: E731
    dt_in = dev(r.standard_normal((*lead, Di)), "f32" if dt32 else dt)
    A = dev(-np.exp(r.uniform(-2, 3, (Di, N))), "f32")
    state = dev(r.standard_normal((slots, Di, N)), "f32")
    kw = dict(D=dev(r.standard_normal(Di), "f32"), z=cut(Di, Di), dt_bias=dev(r.uniform(-7, 0, Di), "f32")) if full else {}
    return cut(0, Di), dt_in, A, cut(2 * Di, N), cut(2 * Di + N + 8, N), state, kw


def check(ops, rows, before, out, after, out_dt, softplus, piece, what):
    x, dt, A, B, C, _, kw = ops
    flat = lambda t: npd(t).reshape(-1, t.shape[-1])[rows]  # noqa: E731
    ref, bound, S, sb = M.scan(flat(x), flat(dt), npd(A), flat(B), flat(C), npd(before), npd(kw.get("D")),
                               flat(kw["z"]) if "z" in kw else None, npd(kw.get("dt_bias")), softplus, piece)
    eo = np.abs(npd(out) - ref) - bound - R.half_ulp(np.abs(ref) + bound, out_dt)
    es = np.abs(npd(after) - S) - sb
    print(f"{what}: {len(ref)} rows, worst out over bound {eo.max() if eo.size else 0:.3g}, state {es.max():.3g}", flush=True)
    assert not eo.size or eo.max() <= 0, what
    assert es.max() <= 0, what


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B,T,Di,dt,dt32,full,softplus,out_dt", [
    (1, 1, 8, "bf16", False, True, True, "bf16"), (3, 1, 200, "f16", True, True, True, "f32"),
    (2, 5, 72, "bf16", True, False, True, "f16"), (4, 2, 40, "f16", False, True, False, "f32"),
])
def test_step(B, T, Di, dt, dt32, full, softplus, out_dt, N):
    ops = draw(B + T + N, (B, T), Di, N, dt, dt32, B + 2, full)
    x, dts, A, Bs, Cs, state, kw = ops
    if not softplus:
        dts.abs_()
        kw.pop("dt_bias", None)
    slots = torch.tensor([*range(1, B + 2, 2), *range(0, B + 2, 2)][:B], dtype=torch.int32).cuda()  # distinct
    before = state.clone()
    out = Q.q1_scan_step(x, dts, A, Bs, Cs, state, slots=slots, softplus=softplus, out_dtype=DT[out_dt], **kw)
    for s in range(B):
        i = int(slots[s])
        check(ops, slice(s * T, (s + 1) * T), before[i], out[s], state[i], out_dt, softplus, 1, f"step N={N} sequence {s}")
    rest = [i for i in range(B + 2) if i not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("lens,Di,N,dt,dt32,full,out_dt", [
    ([1], 8, 16, "bf16", False, True, "f32"), ([77], 136, 16, "f16", False, True, "f16"),
    ([0, 5, 1, 2, 33, 0, 32, 31, 64, 65], 64, 16, "bf16", True, True, "f32"),
    ([200, 0, 15, 129], 72, 8, "bf16", False, False, "bf16"), ([300, 40], 24, 32, "f16", True, True, "f32"),
    ([150, 7], 16, 64, "bf16", False, True, "f32"), ([1] * 60, 16, 16, "f16", False, True, "f32"),
    ([700], 200, 16, "bf16", False, True, "f32"),
])
def test_prefill(lens, Di, N, dt, dt32, full, out_dt):
    """Also the rows before the first and behind the last sequence, which stay as they are."""
    n, lead, tail = sum(lens), 3, 5
    ops = draw(n + Di + N, (lead + n + tail,), Di, N, dt, dt32, len(lens) + 1, full)
    x, dts, A, B, C, state, kw = ops
    cu = torch.tensor(np.cumsum([lead] + lens), dtype=torch.int32).cuda()
    slots = torch.arange(len(lens), 0, -1, dtype=torch.int32).cuda()
    before = state.clone()
    out = torch.full((lead + n + tail, Di), 7.0, dtype=DT[out_dt], device="cuda")
    Q.q1_scan_prefill(x, dts, A, B, C, state, cu, slots=slots, out=out, **kw)
    for s, (t, m) in enumerate(zip(cu.tolist(), lens)):
        i = int(slots[s])
        check(ops, slice(t, t + m), before[i], out[t:t + m], state[i], out_dt, True, PIECE, f"prefill N={N} sequence {s}")
        if m == 0:
            assert torch.equal(state[i], before[i])
    assert (out[:lead] == 7).all() and (out[lead + n:] == 7).all() and torch.equal(state[0], before[0])


def test_many_whole_sequences():
    """More sequences than fill the chip, of a few tokens each: none is cut into pieces."""
    nseq, Di = 520, 512
    lens = [(7 * i) % 5 for i in range(nseq)]
    ops = draw(5, (sum(lens),), Di, 16, "bf16", False, nseq)
    x, dts, A, B, C, state, kw = ops
    before = state.clone()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, out_dtype=torch.float32, **kw)
    for s in (0, 1, 2, 3, 4, 259, 518, 519):
        t = int(cu[s])
        check(ops, slice(t, t + lens[s]), before[s], out[t:t + lens[s]], state[s], "f32", True, PIECE, f"sequence {s}")


def test_one_long_sequence_among_many():
    """Of so many sequences that none need be cut only the one with most of the tokens is; the same rows
    alone, in other pieces, and with no state of its own."""
    nseq, Di = 520, 512
    lens = [(5 * i) % 4 for i in range(nseq)]
    lens[300] = 1700
    ops = draw(12, (sum(lens),), Di, 16, "bf16", False, nseq)
    x, dts, A, B, C, state, kw = ops
    before, alone = state.clone(), state.clone()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, out_dtype=torch.float32, **kw)
    for s in (1, 299, 300, 301, 519):
        t = int(cu[s])
        check(ops, slice(t, t + lens[s]), before[s], out[t:t + lens[s]], state[s], "f32", True, PIECE, f"sequence {s}")
    t = int(cu[300])
    rows = slice(t, t + 1700)
    z, rest = kw["z"], {k: v for k, v in kw.items() if k != "z"}
    one = lambda slot: Q.q1_scan_prefill(x[rows], dts[rows], A, B[rows], C[rows], alone, cu[:1].new_tensor([0, 1700]), z=z[rows],  # noqa: E731
                                         slots=cu[:1].new_tensor([slot]), out_dtype=torch.float32, **rest)
    got = one(300)
    check(ops, rows, before[300], got, alone[300], "f32", True, PIECE, "alone")
    kept = alone.clone()
    assert not one(nseq).any() and torch.equal(alone, kept)


def test_prompt_continues_as_steps_do():
    ops = draw(6, (90,), 48, 16, "f16", False, 2)
    x, dts, A, B, C, state, kw = ops
    before, other = state.clone(), state.clone()
    z, rest = kw["z"], {k: v for k, v in kw.items() if k != "z"}
    cu = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    Q.q1_scan_prefill(x[:50], dts[:50], A, B[:50], C[:50], state, cu(0, 50), z=z[:50], **rest)
    for t in range(50, 90):
        one = slice(t, t + 1)
        out = Q.q1_scan_step(x[None, one], dts[None, one], A, B[None, one], C[None, one], state, z=z[None, one],
                             out_dtype=torch.float32, **rest)
    whole = Q.q1_scan_prefill(x, dts, A, B, C, other, cu(0, 90), z=z, out_dtype=torch.float32, **rest)
    check(ops, slice(0, 90), before[0], whole, other[0], "f32", True, PIECE, "whole")
    ref, bound, S, sb = M.scan(*(npd(v) for v in (x, dts, A, B, C)), npd(before[0]), npd(kw["D"]), npd(z), npd(kw["dt_bias"]),
                               True, PIECE)
    assert (np.abs(npd(state[0]) - S) <= sb).all() and (np.abs(npd(out[0, 0]) - ref[-1]) <= bound[-1] + 2.0 ** -24 * np.abs(ref[-1])).all()


def test_decays_of_zero_and_one():
    """delta A far below -100 forgets exactly, delta = 0 keeps exactly; also softplus far out on both sides."""
    ops = draw(7, (64,), 8, 16, "bf16", True, 1, full=False)
    x, dts, A, B, C, state, kw = ops
    dts[:, 0], dts[:, 1], dts[:, 2], dts[:, 3] = 0.0, 1e4, -200.0, 90.0
    before = state.clone()
    cu = torch.tensor([0, 64], dtype=torch.int32).cuda()
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, softplus=False, out_dtype=torch.float32)
    assert torch.equal(state[0, 0], before[0, 0])  # delta 0: nothing is written, nothing forgotten
    want = 1e4 * npd(x[-1, 1]) * npd(B[-1])
    forgets = npd(A[1]) * 1e4 < -200
    assert forgets.any() and np.allclose(npd(state[0, 1])[forgets], want[forgets], rtol=2.0 ** -22)
    state.copy_(before)
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, out_dtype=torch.float32)
    check(ops, slice(0, 64), before[0], out, state[0], "f32", True, PIECE, "softplus far out")


@pytest.mark.parametrize("T", [1, 90])
def test_nan_and_infinity_stay_in_their_channel(T):
    ops = draw(8, (T,), 32, 16, "bf16", True, 1)
    x, dts, A, B, C, state, kw = ops
    before = state.clone()
    want = Q.q1_scan_prefill(x, dts, A, B, C, state, torch.tensor([0, T], dtype=torch.int32).cuda(), **kw)
    clean = state.clone()
    state.copy_(before)
    at = T // 2
    x[at, 3], dts[at, 4], x[at, 5] = float("nan"), float("nan"), float("inf")
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, torch.tensor([0, T], dtype=torch.int32).cuda(), **kw)
    fine = [c for c in range(32) if c not in (3, 4, 5)]
    assert torch.equal(out[:, fine], want[:, fine]) and torch.equal(state[:, fine], clean[:, fine])
    assert out[at:, 3:5].isnan().all() and state[0, 3:5].isnan().all() and not torch.isfinite(state[0, 5]).any()
    assert torch.equal(out[:at], want[:at])


def test_slots_and_offsets_out_of_range():
    ops = draw(9, (150,), 40, 16, "bf16", False, 2)
    x, dts, A, B, C, state, kw = ops
    before = state.clone()
    cu = torch.tensor([-4, 60, 110, 10 ** 6], dtype=torch.int32).cuda()
    out = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, slots=torch.tensor([-1, 1, 2], dtype=torch.int32).cuda(), **kw)
    assert not out[:60].any() and not out[110:].any() and torch.equal(state[0], before[0])
    check(ops, slice(60, 110), before[1], out[60:110], state[1], "bf16", True, PIECE, "the sequence with a state")
    step = lambda t: t[:3, None]  # noqa: E731
    kw["z"] = step(kw["z"])
    out = Q.q1_scan_step(step(x), step(dts), A, step(B), step(C), state, slots=torch.tensor([5, 0, -2 ** 31], dtype=torch.int32).cuda(), **kw)
    assert not out[[0, 2]].any() and out[1].any()


def test_streams_and_graphs():
    ops = draw(10, (400,), 72, 16, "bf16", False, 2)
    x, dts, A, B, C, state, kw = ops
    cu = torch.tensor([0, 261, 400], dtype=torch.int32).cuda()
    first = state.clone()
    want = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, **kw)
    after = state.clone()
    state.copy_(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(state, after)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state.copy_(first)
        got = Q.q1_scan_prefill(x, dts, A, B, C, state, cu, **kw)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, after)
        other = first.clone()
        Q.q1_scan_prefill(x.clone().mul_(2), dts, A, B, C, other, cu, **kw)


@pytest.mark.parametrize("what", ["dtype", "width", "state", "odd", "host", "dt"])
def test_binding_refusals(what):
    x, dts, A, B, C, state, kw = draw(11, (10,), 64, 16, "bf16", False, 1)
    cu = torch.tensor([0, 10], dtype=torch.int32).cuda()
    if what == "dtype":
        B = B.half()
    elif what == "width":
        C = C[:, :8]
    elif what == "state":
        state = state.double()
    elif what == "odd":
        x, dts, A, state, kw = x[:, :60], dts[:, :60], A[:60].contiguous(), state[:, :60].contiguous(), {}
    elif what == "host":
        kw["D"] = kw["D"].cpu()
    else:
        dts = dts.double()
    with pytest.raises((ValueError, Q.Q1Error)):
        Q.q1_scan_prefill(x, dts, A, B, C, state, cu, **kw)
