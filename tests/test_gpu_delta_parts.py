"""The precision of prompts on the GPU: in fp32 neither the state nor the output is
further from the 64-bit oracle than the recurrent form's over the same tokens, to the
factor that tells two parts of an operand from three."""
import numpy as np
import pytest
import torch

import delta_parts as E
from oracle import decode_oracle as R

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
    return t.double().cpu().numpy()


def operands(seed, T, Hk, Hv, Dk, Dv, dt, rate):
    r = np.random.default_rng(seed)
    n = lambda *s: torch.from_numpy(r.standard_normal(s)).cuda()  # noqa: E731
    q, k, v = (n(T, h, d).to(DT[dt]) for h, d in ((Hk, Dk), (Hk, Dk), (Hv, Dv)))
    g = torch.from_numpy(-r.exponential(1, (T, Hv)) * rate).float().cuda()
    return q, k, v, g, torch.from_numpy(r.uniform(0, 1, (T, Hv))).float().cuda(), 0.3 * n(1, Hv, Dk, Dv).float()


@pytest.mark.parametrize("rate", E.RATES)
@pytest.mark.parametrize("Dk,Dv,dt", [(128, 128, "bf16"), (128, 48, "f16"), (64, 64, "bf16"), (64, 128, "f16")])
def test_prompts_in_fp32(Dk, Dv, dt, rate):
    *x, start = operands(Dk + Dv, 293, 1, 2, Dk, Dv, dt, rate)
    ref, _, S, _ = R.delta_rule(*map(npd, x), npd(start[0]), True, Dk ** -0.5, 1)
    states = [start.clone(), start.clone()]
    step = Q.q1_delta_step(*(a[None] for a in x), states[0], l2norm=True, out_dtype=torch.float32)[0]
    prompt = Q.q1_delta_prefill(*x, states[1], torch.tensor([0, 293], dtype=torch.int32).cuda(), l2norm=True,
                                out_dtype=torch.float32)
    for h in range(2):
        errors = [[E.error(npd(s[0, h]), S[h]) for s in states], [E.error(npd(o[:, h]), ref[:, h]) for o in (step, prompt)]]
        print(f"head {h}: log2 of the error, step and prompt: state {np.log2(errors[0])}, output {np.log2(errors[1])}", flush=True)
        assert errors[0][1] <= E.LIMIT * errors[0][0], "state"
        assert errors[1][1] <= E.LIMIT * errors[1][0], "output"
