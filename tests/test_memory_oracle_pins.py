"""Pins of the oracle of q1_memory.h: hand-worked values and closed forms."""
import numpy as np

from oracle import memory_oracle as M


def test_codes_of_4_bits_by_hand():
    # largest 7: e = 0 (1.75 * 4 = 7); 0.25, 2.5 and 5 are ties and go to the even code, 7 to 6
    x = np.zeros(32)
    x[:9] = [7, -6, 0.25, 2.5, 5, 0.75, -3.4, 1.74, 1e-9]
    c, s = M.kv_encode(x, 4, "bf16")
    assert s.tolist() == [127]
    assert M.kv_decode(c, s, 4)[:9].tolist() == [6, -6, 0, 2, 4, 1, -3, 1.5, 0]
    assert c[:5].tolist() == [7, 15, 0, 4, 6]
    # a little more than 7 doubles the scale
    x[0] = 7.03125
    c, s = M.kv_encode(x, 4, "bf16")
    assert s.tolist() == [128] and M.kv_decode(c, s, 4)[:2].tolist() == [8, -6]


def test_codes_of_8_bits_by_hand():
    x = np.zeros(32)
    x[:6] = [448, -17, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 0.3]
    c, s = M.kv_encode(x, 8, "bf16")
    assert s.tolist() == [127]
    assert M.kv_decode(c, s, 8)[:6].tolist() == [448, -16, 0, 2.0 ** -8, 1.0, 0.3125]
    assert c[0] == 0x7e and c[1] == 0x80 | (11 << 3)


def test_grids_are_the_formats():
    assert len(M.GRID4) == 8 and len(M.GRID8) == 127 and M.GRID8[-1] == 448 and M.GRID8[8] == 2.0 ** -6
    assert (np.diff(M.GRID8) > 0).all()


def test_ends_of_the_scales():
    zero = M.kv_encode(np.zeros(32), 4, "bf16")
    assert zero[1].tolist() == [2] and not zero[0].any()
    top = np.full(32, 65504.0)  # the largest fp16: stays finite in fp16
    for bits, byte, value in ((4, 140, 6 * 2.0 ** 13), (8, 134, 448 * 2.0 ** 7)):
        c, s = M.kv_encode(top, bits, "f16")
        assert s.tolist() == [byte] and (M.kv_decode(c, s, bits) == value).all() and value <= 65504
    big = np.full(32, 255 * 2.0 ** 120)  # the largest bf16
    for bits in (4, 8):
        v = M.kv_decode(*M.kv_encode(big, bits, "bf16"), bits)
        assert (v < 2.0 ** 128).all() and (v >= 0.75 * big).all()
    bad = np.ones(64)
    bad[40] = np.inf
    c, s = M.kv_encode(bad, 8, "bf16")
    assert s[1] == 255 and not c[32:].any() and np.isnan(M.kv_decode(c, s, 8)[32:]).all()


def test_round_trip_is_idempotent_and_within_half_a_step():
    r = np.random.default_rng(1)
    x = r.standard_normal((50, 64)) * np.exp(r.uniform(-8, 8, (50, 1)))
    # a code has m = 1 or 3 bits behind its leading one: a value is at most half a step off, relatively
    # most at the tie after a power of two, 1 + 2^-(m+1) of it: by 2^-(m+1) / (1 + 2^-(m+1)) = 1/5 or 1/17,
    # and no element is larger than the largest
    for bits, off in ((4, 1 / 5), (8, 1 / 17)):
        v = M.kv_decode(*M.kv_encode(x, bits, "bf16"), bits)
        again = M.kv_decode(*M.kv_encode(v, bits, "bf16"), bits)
        assert (np.abs(v - x).max(1) <= off * np.abs(x).max(1)).all()
        assert (v == again).all()
        assert (M.unpack(M.pack(M.kv_encode(x, bits, "bf16")[0], bits), bits) == M.kv_encode(x, bits, "bf16")[0]).all()


def test_convolution_by_hand():
    # taps 1, 10, 100 over 1, 2 | 3, 4, 5
    out, _, state = M.conv([[3.0], [4], [5]], [[1.0, 10, 100]], [0.5], [[1.0], [2]], False)
    assert out[:, 0].tolist() == [321.5, 432.5, 543.5] and state[:, 0].tolist() == [4, 5]
    out, _, state = M.conv([[3.0]], [[0.0, 0, 1]], None, [[1.0], [2]], True)
    assert np.allclose(out, 3 / (1 + np.exp(-3.0))) and state[:, 0].tolist() == [2, 3]


def test_scan_by_hand():
    # delta = 2, A = -log 2: a = 1/4; h = 8/4 + 2*3*0.5 = 5; y = 5*2 + 3*10; gate 0 halves nothing: silu(0) = 0
    out, _, h, _ = M.scan([[3.0]], [[2.0]], [[-np.log(2)]], [[0.5]], [[2.0]], [[8.0]], D=[10.0], softplus=False)
    assert np.allclose(h, 5.0) and np.allclose(out, 40.0)
    out, _, _, _ = M.scan([[3.0]], [[2.0]], [[-np.log(2)]], [[0.5]], [[2.0]], [[8.0]], z=[[0.0]], softplus=False)
    assert (out == 0).all()
    # softplus(0) = log 2
    _, _, h, _ = M.scan([[1.0]], [[1.0]], [[0.0]], [[1.0]], [[1.0]], [[0.0]], dt_bias=[-1.0])
    assert np.allclose(h, np.log(2))


def test_scan_of_constant_input_reaches_its_limit():
    # h = a h + d b x tends to d b x / (1 - a)
    n = 2000
    one = np.ones((n, 1))
    _, _, h, e = M.scan(one, 0.1 * one, [[-1.0]], one, one, [[0.0]], softplus=False)
    assert np.allclose(h, 0.1 / (1 - np.exp(-0.1))) and (e < 1e-4).all()
