"""Attention over quantised pages whose values are near the largest of their type: a weighted mean
of them is no larger than they are, however many tokens it is of and wherever the maximum of
the scores is first met.  Against the 64-bit oracle; tolerances are its bounds, the
output's rounding, and weights that become 0: of n tokens those below n 2^-117 of the largest (they
are relative to 2^8 2^bits(n) times a maximum that may be 2^8 below the true one, and 2^bits(n) is at
most 2 n; below 2^-126 they are 0), n of them, each times the largest value."""
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


def run(keys, values, q, bits, page=16, room=0, scale=None):
    """keys, values [n, Hkv, D] and q [T, Hq, D] bf16 on the CPU; returns (out, lse, held keys, held values)."""
    n, Hkv, D = keys.shape
    per = -(-n // page)
    cache = Q.PackedKV.empty(per + 1, page, Hkv, D, bits)
    table = torch.randperm(per, generator=torch.Generator().manual_seed(n)).int()
    slots = (table.repeat_interleave(page)[:n] * page + torch.arange(n, dtype=torch.int32) % page).cuda()
    Q.q1_kv_write(cache, keys.cuda(), values.cuda(), slots.int())
    wide = torch.zeros(1, max(per, room // page), dtype=torch.int32)
    wide[0, :per] = table
    out, lse = Q.q1_kv_attn(q[None].cuda(), cache, wide.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), scale=scale,
                            out_dtype=torch.float32)
    held = [npd(x) for x in Q.q1_kv_read(cache, slots.int(), torch.float32)]
    return npd(out[0]), npd(lse[0]), held[0], held[1]


def check(out, lse, k, v, q, some, scale=None):
    T, D = q.shape[0], q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    for t in some:
        m = len(k) - (T - 1 - t)
        ref, bound, l, lb = R.prefix_attention(npd(q[t]), k[:m], v[:m], scale)
        bound = bound + m * m * 2.0 ** -117 * np.abs(v[:m]).max()
        assert np.isfinite(out[t]).all(), t
        assert (np.abs(out[t] - ref) <= bound + R.half_ulp(np.abs(ref) + bound, "f32")).all(), t
        assert (np.abs(lse[t] - l) <= lb).all(), t


# (prompts of 1024 queries for 32 heads of keys are done by rows)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,T,Hq,Hkv,D,room", [(300, 1, 4, 2, 64, 0), (1, 1, 2, 2, 128, 0), (5000, 1, 8, 1, 128, 0), (700, 3, 12, 2, 256, 0),
                                               (40000, 2, 2, 1, 64, 0), (1100, 1024, 32, 32, 64, 4096), (1024, 1024, 16, 16, 256, 4096)])
def test_the_largest_values(n, T, Hq, Hkv, D, room, bits):
    """All values as large as pages hold them: so is their mean, to the weights' rounding."""
    r = torch.Generator().manual_seed(n)
    k, q = torch.randn(n, Hkv, D, generator=r).bfloat16(), torch.randn(T, Hq, D, generator=r).bfloat16()
    v = torch.full((n, Hkv, D), 3.3e38).bfloat16()
    v[..., 1::2] *= -1
    out, lse, hk, hv = run(k, v, q, bits, room=room)
    assert (np.abs(hv) >= 1.5 * 2.0 ** 127).all()
    check(out, lse, hk, hv, q, sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,Hkv,room", [(1, 1, 0), (4, 2, 0), (1024, 32, 4096)])
@pytest.mark.parametrize("first,second", [(2.0 ** 121, 2.0 ** 121), (2.0 ** 121, 1.0), (1.0, 2.0 ** 121), (2.0 ** 88, -2.0 ** 126)])
def test_a_maximum_that_stays_in_place(first, second, T, Hkv, room, bits):
    """Scores that rise by 7 powers of two from one tile to the next: the old maximum is kept."""
    D, n = 64, max(T, 256) + 40
    k = torch.zeros(n, Hkv, D)
    k[128:] = 1.0
    k[n - 20:] = 0.5
    v = torch.full((n, Hkv, D), first)
    v[128:] = second
    q = torch.ones(T, Hkv, D).bfloat16()
    scale = 7 * np.log(2.0) / D
    out, lse, hk, hv = run(k.bfloat16(), v.bfloat16(), q, bits, room=room, scale=scale)
    check(out, lse, hk, hv, q, sorted({0, T // 2, T - 1}), scale=np.float64(np.float32(scale)))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("seed,n,T,Hq,Hkv,D,room", [(1, 900, 1, 6, 2, 64, 0), (2, 20000, 2, 12, 1, 128, 0), (3, 3000, 1, 4, 1, 256, 0),
                                                    (4, 1200, 1024, 32, 32, 128, 4096)])
def test_a_few_large_values(seed, n, T, Hq, Hkv, D, room, bits):
    """Ordinary values, and some tokens' from 2^80 to the largest, some of them behind what early queries see."""
    r = np.random.default_rng(seed)
    k = torch.from_numpy(2 * r.standard_normal((n, Hkv, D))).bfloat16()
    v = r.standard_normal((n, Hkv, D))
    for i in [*r.integers(0, n, 6), n - 1, n - 2]:
        v[i] = np.clip(v[i], -1.9, 1.9) * 2.0 ** r.integers(80, 127)
    q = torch.from_numpy(2 * r.standard_normal((T, Hq, D))).bfloat16()
    out, lse, hk, hv = run(k, torch.from_numpy(v).bfloat16(), q, bits, page=64, room=room)
    check(out, lse, hk, hv, q, sorted({0, T // 2, max(0, T - 2), T - 1}))


@pytest.mark.parametrize("T,Hkv,room", [(1, 1, 0), (1024, 32, 4096)])
def test_the_largest_scale(T, Hkv, room):
    """Scores of 0 are 0 at any scale: a row is the mean of what it sees."""
    D, n = 64, max(T, 70)
    k, v = torch.ones(n, Hkv, D).bfloat16(), torch.arange(n).remainder(7)[:, None, None].expand(n, Hkv, D).bfloat16()
    q = torch.zeros(T, Hkv, D).bfloat16()
    for scale in (3.4e38, -3.4e38, 1e-45):
        out, lse, hk, hv = run(k, v, q, 8, room=room, scale=scale)
        check(out, lse, hk, hv, q, sorted({0, T // 2, T - 1}), scale=scale)
