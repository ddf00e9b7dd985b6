"""Pins of the decode-step oracle: hand-worked values and closed forms."""
import numpy as np

from oracle import decode_oracle as R


def test_delta_rule_by_hand():
    # one head, Dk = Dv = 1 twice over: S = 2, a = 1/2, k = 1, beta = 1/2, v = 3:
    # S' = 1 + 1/2 (3 - 1) = 2, o = 2 * 5 * 0.1
    out, _, S, _ = R.delta_rule([[[5.0]]], [[[1.0]]], [[[3.0]]], [[np.log(0.5)]], [[0.5]], [[[2.0]]], False, 0.1, 1)
    assert np.allclose(S, 2.0) and np.allclose(out, 1.0)


def test_delta_rule_writes_and_reads_back():
    # beta = 1, g = 0, orthonormal keys: reading key i gives value i; writing it again replaces it
    k = np.eye(4)[:, None, :]
    v = np.arange(8.0).reshape(4, 1, 2)
    zero, one = np.zeros((4, 1)), np.ones((4, 1))
    _, _, S, _ = R.delta_rule(k, k, v, zero, one, np.zeros((1, 4, 2)), False, 1.0, 1)
    assert np.allclose(S[0], v[:, 0])
    out, _, S, _ = R.delta_rule(k[:1], k[:1], [[[9.0, 9.0]]], zero[:1], one[:1], S, False, 1.0, 1)
    assert np.allclose(out, 9.0) and np.allclose(S[0, 0], 9.0) and np.allclose(S[0, 1:], v[1:, 0])


def test_delta_rule_forgets_exactly():
    _, _, S, e = R.delta_rule([[[0.0]]], [[[0.0]]], [[[1.0]]], [[-np.inf]], [[1.0]], [[[7.0]]], False, 1.0, 1)
    assert S[0, 0, 0] == 0.0


def test_attention_by_hand():
    # two equal scores average the values; a third token 1000 below adds nothing
    keys = np.array([[[1.0, 0]], [[1.0, 0]], [[-999.0, 0]]])
    out, _, lse, _ = R.prefix_attention([[1.0, 0.0]], keys, np.array([[[2.0, 0]], [[4.0, 0]], [[50.0, 1]]]), 1.0)
    assert np.allclose(out, [[3.0, 0.0]]) and np.allclose(lse, 1.0 + np.log(2))


def test_attention_of_nothing():
    out, _, lse, _ = R.prefix_attention(np.ones((2, 4)), np.zeros((0, 1, 4)), np.zeros((0, 1, 4)), 1.0)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_half_ulp():
    assert R.half_ulp(np.array([1.0, 1.5, 2.0]), "bf16").tolist() == [2.0 ** -8, 2.0 ** -8, 2.0 ** -7]
    assert R.half_ulp(np.array([0.0]), "f16")[0] == 2.0 ** -25


def test_sample_by_hand():
    row = np.log(np.array([1.0, 2.0, 4.0, 1.0])).astype(np.float32)
    assert [R.sample(row, u)[0] for u in (0.0, 0.124, 0.13, 0.37, 0.38, 0.87, 0.88)] == [0, 0, 1, 1, 2, 2, 3]
    assert np.isclose(R.sample(row, 0.5)[1], np.log(0.5))
    assert [R.sample(row, u, top_k=2)[0] for u in (0.0, 0.32, 0.34)] == [1, 1, 2]
    assert [R.sample(row, u, top_k=3)[0] for u in (0.0, 0.99)] == [0, 2]      # of equal logits the first is kept
    assert [R.sample(row, u, top_p=0.45)[0] for u in (0.0, 0.99)] == [2, 2]
    assert [R.sample(row, u, top_p=0.55)[0] for u in (0.0, 0.99)] == [1, 2]
    assert [R.sample(row, u, min_p=0.4)[0] for u in (0.0, 0.99)] == [1, 2]
    assert R.sample(row, 0.99, temperature=0.0)[:2] == (2, 0.0)
    assert R.sample(row, 0.99, temperature=1e-3)[0] == 2


def test_sample_edges():
    inf = np.inf
    assert R.sample([-inf, np.nan], 0.5)[:2] == (-1, -inf)
    assert R.sample([np.nan, -5.0, -inf], 0.9)[0] == 1
    assert [R.sample([inf, 3.0, inf], u)[0] for u in (0.4, 0.6)] == [0, 2]
    assert R.sample([0.0, 0.0], 1.0)[0] == 1 and R.sample([0.0, 0.0], -1.0)[0] == 0
    assert R.sample([0.0, 1.0], 0.99, top_p=0.0)[0] == 1 and R.sample([0.0, 1.0], 0.99, min_p=7.0)[0] == 1


def test_sample_choices():
    # the draw 1e-8 past the boundary of two tokens of which one is not exact: either; of two exact ones: the one
    row = np.array([0.0, 0.0, -1.0], np.float32)
    W = 2 + np.exp(-1.0)
    assert {t for t, _ in R.sample_choices(row, (2 + 1e-8) / W)} == {1, 2}
    assert {t for t, _ in R.sample_choices(row[:2], 0.5)} == {1}
    assert {t for t, _ in R.sample_choices(row, 0.2)} == {0}
