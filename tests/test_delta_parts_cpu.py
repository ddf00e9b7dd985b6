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
