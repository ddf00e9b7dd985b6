"""How many parts the chunked delta rule's operands need (no GPU): three reach the
recurrence's own precision in fp32, two do not, in the state and in the output."""
import numpy as np
import pytest

import delta_parts as E
from oracle import decode_oracle as R


def operands(seed, rate, T=256, D=128):
    r = np.random.default_rng(seed)
    q, k, v = (E.nearest(r.standard_normal((T, D)).astype(np.float32)) for _ in range(3))
    return (q, k, v, -(r.exponential(1, T) * rate).astype(np.float32), r.uniform(0, 1, T).astype(np.float32),
            (0.3 * r.standard_normal((D, D))).astype(np.float32))


@pytest.mark.parametrize("rate", E.RATES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_three_parts_and_no_fewer(seed, rate):
    x, scale = operands(seed, rate), 128 ** -0.5
    ref, _, S, _ = R.delta_rule(*(a[:, None] for a in x[:5]), x[5][None], True, scale, 1)
    ref, S = ref[:, 0], S[0]
    limit = [E.LIMIT * E.error(*p) for p in zip(E.recurrent(*x, scale), (ref, S))]

    def over(**kw):
        return [E.error(*p) > most for *p, most in zip(E.chunked(*x, scale, **kw), (ref, S), limit)]

    assert over() == [False, False]
    assert over(out_parts=2) == [True, False]
    assert over(state_parts=2) == [True, True]


@pytest.mark.parametrize("kind", ["random", "all ones"])
def test_what_16_bit_outputs_leave_out(kind):
    """Sums of products of two fp32 operands in two parts each, as outputs in 16 bits have them: with bf16
    operands below 2^-13 of the terms' magnitudes (no product of the low parts), with fp16 ones below 2^-15
    (low parts to the nearest, all products)."""
    r = np.random.default_rng(4)
    bits = r.integers(0, 1 << 23, (2, 4000, 64)) if kind == "random" else np.full((2, 1, 64), (1 << 23) - 1)
    x, y = ((b | 127 << 23).astype(np.uint32).view(np.float32) * r.choice([-1, 1], b.shape).astype(np.float32)
            for b in bits)
    exact, size = x.astype(np.float64) * y, np.abs(x.astype(np.float64) * y)

    def two(a, low):
        high = E.cut(a)
        return high.astype(np.float64), low(a - high).astype(np.float64)

    (v0, v1), (p0, p1) = two(x, E.cut), two(y, E.nearest)
    left = np.abs((v0 * p0 + v0 * p1 + v1 * p0 - exact).sum(-1)) / size.sum(-1)
    worst = (np.abs(v0 * p0 + v0 * p1 + v1 * p0 - exact) / size).max()
    assert left.max() < 2.0 ** -13 and worst < 2.0 ** -13 and (kind == "random" or worst > 2.0 ** -16)
    (v0, v1), (p0, p1) = two(x, E.nearest), two(y, E.nearest)
    assert (np.abs((v0 + v1) * (p0 + p1) - exact) / size).max() < 2.0 ** -15
    (s0, s1) = two(x, E.cut)
    assert (np.abs(s0 + s1 - x) / np.abs(x)).max() < 2.0 ** -15
