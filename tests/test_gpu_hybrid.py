"""The operators together: a small hybrid decoder whose prompt goes through the
chunked and whose decode steps go through the recurrent and paged forms."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q
    from gemm_decode_q1_amd.hybrid import HybridDecoder


@pytest.fixture(scope="module")
def model():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield HybridDecoder(pattern="dad", hidden=512, inter=1024, vocab=1500, Hk=2, Hv=4, Hq=4, Hkv=2, seed=3)
    torch.cuda.synchronize()


def ids_of(model, n, seed):
    return torch.randint(0, model.vocab, (n,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def far(a, b):
    return ((a - b).norm(dim=-1) / b.norm(dim=-1)).max().item()


@pytest.mark.parametrize("P,more", [(1, 3), (70, 20), (129, 35)])
def test_steps_continue_the_prompt(model, P, more):
    """Feeding tokens one by one gives the logits of the longer prompt.  Both forms
    round to bf16 (2^-9 of a value) at about 8 places a layer, 3 layers and the head:
    in the worst case 25 of them add, 25/512; a wrong state or page is off by order one."""
    ids = ids_of(model, P + more, P)
    want = [model.prompt(ids[:n + 1]) for n in range(P, P + more)]
    model.prompt(ids[:P])
    model.begin(3, more)
    for n in range(more):
        got = model.logits(ids[P + n].repeat(3))
        assert far(got, want[n].expand(3, -1)) <= 25 / 512


def test_generate(model):
    """Every answer is as long as asked and drawn from the vocabulary; a captured
    step gives the tokens of the eager one, also when other calls run between; the
    log-probabilities of greedy answers are zero."""
    ids, B, n = ids_of(model, 90, 1), 5, 40
    filters = dict(temperature=torch.linspace(0.5, 1.5, B).cuda(), top_p=torch.full((B,), 0.9).cuda())
    eager = model.generate(ids, B, n, seed=4, graph=False, **filters)
    for _ in range(2):
        got = model.generate(ids, B, n, seed=4, **filters)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
    assert eager[0].shape == (B, n) and int(eager[0].min()) >= 0 and int(eager[0].max()) < model.vocab
    assert len({tuple(t) for t in eager[0].tolist()}) == B
    tokens, logprob = model.generate(ids, 2, 10, temperature=torch.zeros(2).cuda())
    assert torch.equal(tokens[0], tokens[1]) and not logprob.any()


def test_workspace_of_a_captured_call(model):
    """A captured call keeps its workspace while eager calls need ever larger ones."""
    V = 4096
    x = torch.randn(2, V, generator=torch.Generator().manual_seed(2)).cuda()
    u, p = torch.tensor([0.3, 0.8]).cuda(), torch.tensor([0.9, 0.5]).cuda()
    want = [t.clone() for t in Q.q1_sample(x, u, top_p=p)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = Q.q1_sample(x, u, top_p=p)
    for B in (8, 64, 200):
        Q.q1_sample(torch.randn(B, V, device="cuda"), torch.rand(B, device="cuda"), top_p=torch.full((B,), 0.9, device="cuda"))
        torch.randn(1 << 22, device="cuda")
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
