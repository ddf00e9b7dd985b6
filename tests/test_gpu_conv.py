"""The short causal convolution on the GPU against the 64-bit oracle: single tokens and
prompts, widths and types, ragged and empty sequences, slots outside the pool, rows of
no sequence, strided operands, NaN and infinities, streams, graph replays."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as R
from oracle import memory_oracle as M

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield
    torch.cuda.synchronize()


def npd(t):
    return t.detach().double().cpu().numpy()


def draw(seed, rows, C, W, dt, slots, bias=True, strided=True):
    r = np.random.default_rng(seed)
    dev = lambda a: torch.from_numpy(a).to(DT[dt]).cuda()  # noqa: E731
    x = dev(2 * r.standard_normal((rows, C + (24 if strided else 0))))[:, 8 if strided else 0:][:, :C]
    return (x, dev(r.standard_normal((C, W))), dev(r.standard_normal((slots, W - 1, C))),
            dev(r.standard_normal(C)) if bias else None)


def check(x, weight, bias, before, out, after, silu, dt, what):
    """One sequence: the window is exact, outputs within the bound and half a step."""
    ref, bound, state = M.conv(npd(x), npd(weight), None if bias is None else npd(bias), npd(before), silu)
    over = np.abs(npd(out) - ref) - bound - R.half_ulp(np.abs(ref) + bound, dt)
    print(f"{what}: {len(ref)} rows, worst over bound {over.max() if over.size else 0:.3g}", flush=True)
    assert not over.size or over.max() <= 0
    assert np.array_equal(npd(after), state)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C,dt,bias,silu", [(1, 1, 8, "bf16", False, True), (3, 1, 1048, "f16", True, True),
                                                (5, 2, 64, "bf16", True, False), (2, 7, 200, "f16", False, True)])
def test_step(B, T, C, dt, bias, silu, W):
    x, w, state, b = draw(B + T + C, B * T, C, W, dt, B + 2, bias)
    slots = torch.tensor([*range(1, B + 2, 2), *range(0, B + 2, 2)][:B], dtype=torch.int32).cuda()  # distinct
    before = state.clone()
    out = Q.q1_conv_step(x.unflatten(0, (B, T)), w, state, b, slots, silu)
    for s in range(B):
        i = int(slots[s])
        check(x[s * T:(s + 1) * T], w, b, before[i], out[s], state[i], silu, dt, f"step W={W} sequence {s}")
    rest = [i for i in range(B + 2) if i not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens,C,dt", [([1], 8, "bf16"), ([77], 264, "f16"), ([0, 5, 1, 2, 3, 0, 16, 17, 33], 64, "bf16"),
                                       ([200, 0, 15], 520, "bf16"), ([1] * 40, 16, "f16")])
def test_prefill(lens, C, dt, W):
    """Also the rows before the first and behind the last sequence, which stay as they are."""
    n, lead, tail = sum(lens), 3, 5
    x, w, state, b = draw(n + C, lead + n + tail, C, W, dt, len(lens) + 1)
    cu = torch.tensor(np.cumsum([lead] + lens), dtype=torch.int32).cuda()
    slots = torch.arange(len(lens), 0, -1, dtype=torch.int32).cuda()
    before = state.clone()
    out = torch.full((lead + n + tail, C), 7.0, dtype=DT[dt], device="cuda")
    Q.q1_conv_prefill(x, w, state, cu, b, slots, out=out)
    for s, (t, m) in enumerate(zip(cu.tolist(), lens)):
        i = int(slots[s])
        check(x[t:t + m], w, b, before[i], out[t:t + m], state[i], True, dt, f"prefill W={W} sequence {s}")
    assert (out[:lead] == 7).all() and (out[lead + n:] == 7).all() and torch.equal(state[0], before[0])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prompts_and_steps_give_the_same_bits(dt):
    x, w, state, b = draw(11, 90, 136, 4, dt, 2)
    other, third = state.clone(), state.clone()
    cu = torch.tensor([0, 90], dtype=torch.int32).cuda()
    whole = Q.q1_conv_prefill(x, w, state, cu, b)
    steps = torch.cat([Q.q1_conv_step(x[None, t:t + 1], w, other, b)[0] for t in range(90)])
    cut = torch.cat([Q.q1_conv_prefill(x[a:z], w, third, torch.tensor([0, z - a], dtype=torch.int32).cuda(), b)
                     for a, z in ((0, 1), (1, 38), (38, 90))])
    for got, s in ((steps, other), (cut, third)):
        assert torch.equal(got, whole) and torch.equal(s, state)


def test_slots_and_offsets_out_of_range():
    x, w, state, b = draw(12, 30, 40, 3, "bf16", 2)
    before = state.clone()
    cu = torch.tensor([-4, 10, 20, 10 ** 6], dtype=torch.int32).cuda()
    out = Q.q1_conv_prefill(x, w, state, cu, b, torch.tensor([-1, 1, 2], dtype=torch.int32).cuda())
    assert not out[:10].any() and not out[20:].any() and torch.equal(state[0], before[0])
    check(x[10:20], w, b, before[1], out[10:20], state[1], True, "bf16", "the sequence with a state")
    out = Q.q1_conv_step(x[:3, None], w, state, b, torch.tensor([5, 0, -2 ** 31], dtype=torch.int32).cuda())
    assert not out[[0, 2]].any() and out[1].any()


def test_nan_and_infinity_stay_where_they_are():
    x, w, state, _ = draw(13, 20, 32, 4, "bf16", 1, strided=False)
    w = w.abs() + 0.1
    state.zero_()
    x[5, 3], x[9, 4], x[9, 5], x[12, 6] = float("nan"), float("inf"), -float("inf"), -3e38
    out = Q.q1_conv_prefill(x, w, state, torch.tensor([0, 20], dtype=torch.int32).cuda())
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[5:9, 3] = want[9:13, 4] = want[9:13, 5] = True
    # sums are fp32: -3e38 w is -infinity for w > 1.134, and s / (1 + exp(-s)) of that a NaN
    want[12:16, 6] = torch.isinf(x[12, 6].float() * w[6].flip(0).float())
    assert torch.equal(bad, want) and out[5:9, 3].isnan().all() and (out[9:13, 4] == float("inf")).all()


def test_large_arguments_of_the_activation():
    """silu of sums far below and above zero, where exp(-s) overflows and underflows."""
    C = 64
    x = torch.linspace(-300, 300, 128 * C).view(128, C).bfloat16().cuda()
    w = torch.zeros(C, 4).bfloat16().cuda()
    w[:, 3] = 1
    state = torch.zeros(1, 3, C).bfloat16().cuda()
    before = state.clone()
    out = Q.q1_conv_prefill(x, w, state, torch.tensor([0, 128], dtype=torch.int32).cuda())
    check(x, w, None, before[0], out, state[0], True, "bf16", "large arguments")


def test_streams_and_graphs():
    x, w, state, b = draw(14, 100, 72, 4, "f16", 3)
    cu = torch.tensor([0, 61, 100], dtype=torch.int32).cuda()
    first = state.clone()
    want = Q.q1_conv_prefill(x, w, state, cu, b)
    after = state.clone()
    side = torch.cuda.Stream()
    state.copy_(first)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = Q.q1_conv_prefill(x, w, state, cu, b)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(state, after)
    token = x[:3, None].contiguous()
    graph = torch.cuda.CUDAGraph()
    state.copy_(first)
    with torch.cuda.graph(graph):
        got = Q.q1_conv_step(token, w, state, b)
    other = first.clone()
    state.copy_(first)
    for i in range(4):
        token.normal_()
        graph.replay()
        want = Q.q1_conv_step(token, w, other, b)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, other)


@pytest.mark.parametrize("what", ["dtype", "width", "state", "odd", "host", "cu"])
def test_binding_refusals(what):
    x, w, state, b = draw(15, 10, 64, 4, "bf16", 1)
    cu = torch.tensor([0, 10], dtype=torch.int32).cuda()
    if what == "dtype":
        w = w.half()
    elif what == "width":
        w = torch.zeros(64, 5, device="cuda", dtype=torch.bfloat16)
    elif what == "state":
        state = state[:, :2]
    elif what == "odd":
        x = x[:, :60]
    elif what == "host":
        b = b.cpu()
    else:
        cu = cu.long()
    with pytest.raises((ValueError, Q.Q1Error)):
        Q.q1_conv_prefill(x, w, state, cu, b)
