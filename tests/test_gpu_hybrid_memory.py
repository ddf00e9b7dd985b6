"""What a decoder remembers, together: convolution, scan and delta rule, keys and
values in quantised pages.  A prompt goes through the packed forms, decode steps
through the forms for single tokens; the prompt's pages are shared by the batch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q
    from gemm_decode_q1_amd.hybrid import HybridDecoder


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    yield
    torch.cuda.synchronize()


def build(pattern, conv, bits, seed=3):
    return HybridDecoder(pattern=pattern, hidden=512, inter=1024, vocab=1500, Hk=2, Hv=4, Hq=4, Hkv=2, seed=seed, conv=conv,
                         kv_bits=bits, channels=768, N=16)


def ids_of(model, n, seed):
    return torch.randint(0, model.vocab, (n,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def far(a, b):
    return ((a - b).norm(dim=-1) / b.norm(dim=-1)).max().item()


@pytest.mark.parametrize("pattern,conv,bits", [("sds", 4, 16), ("ss", 0, 16), ("dd", 2, 16), ("saa", 3, 8), ("das", 4, 4)])
@pytest.mark.parametrize("P,more", [(1, 3), (64, 18), (129, 35)])
def test_steps_continue_the_prompt(pattern, conv, bits, P, more):
    """Feeding tokens one by one gives the logits of the longer prompt.  Both forms round to bf16
    (2^-9 of a value) at about 8 places a layer and one more for a convolution, 3 layers and
    the head: in the worst case d = 28 of them add, 28/512.  Keys and values that differ by d
    go to another code, a step s of the value away (s at most 1/8 in 8 bits, 1/2 in 4), for d / s
    of them: in the mean square sqrt(d s), of keys and of values, for each layer of attention.
    A wrong state, row or page is off by order one."""
    model = build(pattern, conv, bits)
    d = 28 / 512
    most = d + (0 if bits == 16 else pattern.count("a") * 2 * (d * {8: 1 / 8, 4: 1 / 2}[bits]) ** 0.5)
    ids = ids_of(model, P + more, P)
    want = {n: model.prompt(ids[:n + 1]) for n in (P, P + 1, P + more - 1)}
    model.prompt(ids[:P])
    model.begin(3, more)
    for n in range(P, P + more):
        got = model.logits(ids[n].repeat(3))
        if n in want:
            print(pattern, bits, n, "off by", far(got, want[n].expand(3, -1)), "of", most, flush=True)
            assert far(got, want[n].expand(3, -1)) <= most


def test_answers_of_a_batch_do_not_meet():
    """Sequences that share the prompt's pages and go on with other tokens: each has the logits
    that it has alone, bit for bit (the same forms run on more rows)."""
    model = build("das", 4, 4)
    ids = ids_of(model, 70, 9)
    model.prompt(ids)
    tokens = ids_of(model, 24, 10).view(3, 8)
    model.begin(3, 8)
    together = [model.logits(tokens[:, t].contiguous()) for t in range(8)]
    for b in range(3):
        model.begin(3, 8)
        for t in range(8):
            alone = model.logits(tokens[b, t].repeat(3))
            assert torch.equal(alone[b], together[t][b]), (b, t)


@pytest.mark.parametrize("pattern,conv,bits", [("dsa", 4, 4), ("sa", 2, 8)])
def test_generate(pattern, conv, bits):
    """A captured step gives the tokens of the eager one, also when other calls run between."""
    model = build(pattern, conv, bits)
    ids, B, n = ids_of(model, 90, 1), 5, 30
    filters = dict(temperature=torch.linspace(0.5, 1.5, B).cuda(), top_p=torch.full((B,), 0.9).cuda())
    eager = model.generate(ids, B, n, seed=4, graph=False, **filters)
    for _ in range(2):
        got = model.generate(ids, B, n, seed=4, **filters)
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
    assert eager[0].shape == (B, n) and int(eager[0].min()) >= 0 and int(eager[0].max()) < model.vocab
    assert len({tuple(t) for t in eager[0].tolist()}) == B


@pytest.mark.parametrize("bits", [4, 8])
def test_quantised_pages_are_near_the_16_bit_ones(bits):
    """Half a step of keys and of values (1/16 of a value in 8 bits, at most 1/4 in 4) in one layer,
    next to the 28 roundings of 2^-9 of the rest."""
    ids = None
    logits = []
    for b in (16, bits):
        model = build("da", 0, b, seed=5)
        ids = ids_of(model, 140, 3) if ids is None else ids
        logits.append(model.prompt(ids))
    assert 0 < far(logits[1], logits[0]) <= 28 / 512 + 2 * {8: 1 / 16, 4: 1 / 4}[bits]
