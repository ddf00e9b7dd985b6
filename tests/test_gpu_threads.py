"""Calls of several threads on one stream: each gets the results that it gets alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield
    torch.cuda.synchronize()


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    T, P, V = 200, 900, 9000
    prompt = (r(T, 1, 64).bfloat16(), r(T, 1, 64).bfloat16(), r(T, 2, 64).bfloat16(), -r(T, 2).exp(), r(T, 2).sigmoid())
    attn = (r(3, 4, 64).bfloat16(), r(P, 2, 64).bfloat16(), r(P, 2, 64).bfloat16())
    rows = (3 * r(3, V), torch.rand(3, generator=g).cuda(), torch.full((3,), 0.9).cuda())
    return prompt, r(1, 2, 64, 64), torch.tensor([0, T], dtype=torch.int32).cuda(), attn, rows


def results(prompt, state, cu, attn, rows):
    state = state.clone()
    out = Q.q1_delta_prefill(*prompt, state, cu, l2norm=True)
    return [out, state, *Q.q1_prefix_attn(*attn), *Q.q1_sample(rows[0], rows[1], top_p=rows[2])]


def test_threads_on_one_stream():
    n, repeats = 3, 40
    given = [inputs(i) for i in range(n)]
    want = [[x.clone() for x in results(*g)] for g in given]
    torch.cuda.synchronize()
    got = [[] for _ in range(n)]

    def work(i):
        for _ in range(repeats):
            got[i].append(results(*given[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(n):
        assert len(got[i]) == repeats
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))
