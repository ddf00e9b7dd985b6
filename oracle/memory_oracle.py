"""CPU oracle of the calls of ``include/q1_memory.h``: NumPy, 64 bits, straight from
the definitions there.  Shares no code with the HIP path.  Attention over the
values that pages hold is ``decode_oracle.prefix_attention``, with its bound.

Error bounds beside the values, u = 2^-24 being half a step of fp32:

* ``conv``: a sum of W products and a bias, by multiply-adds: (W + 1) u of the sum of
  the absolute terms.  silu(s) = s / (1 + E), E = exp(-s): the argument of the
  exponential is off by (2 |s|) u, so E by (2 |s| + 2) u, the quotient by that times
  E / (1 + E) <= 1, and sum, reciprocal and product by 4 u: |silu(s)| (2 |s| + 6) u.  Its
  slope is below 1.1.  (Where E overflows the value is 0, off by less than 1e-36.)
* ``scan``: delta is softplus(s), s off by |s| u and, in the exponential, by a quarter of that more:
  by sigmoid(s) 1.25 |s| u + 16 u delta (an exponential within 3 u, some multiply-adds of falling
  weight, a reciprocal and four roundings).
  a = exp(delta A) is off by a factor within |A| e_delta + |delta A| (3 + n) u + 2 u: A log2(e)
  and the product are rounded, and over a piece of n tokens the deltas are summed.
  A state's error obeys e' = a e + |a h| (that + 2 u) + |delta x B| (e_delta / delta + 3 u);
  the output adds sum |C| e + (N + 4) u (sum |C h| + |D x|), times the gate, whose own error is
  that of silu.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
GRID4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
GRID8 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
RANGE = {(4, "bf16"): (2, 252), (4, "f16"): (2, 140), (8, "bf16"): (10, 246), (8, "f16"): (10, 134)}


def kv_encode(x, bits, dt):
    """x [..., D] of a 16-bit type: (codes [..., D], scale bytes [..., D / 32])."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 32)
    grid, p = (GRID4, 2) if bits == 4 else (GRID8, 8)
    top = np.abs(y).max(-1)
    finite = np.isfinite(y).all(-1)
    m, ex = np.frexp(np.where(finite, top, 0))           # m in [0.5, 1)
    e = np.where(2 * m > 1.75, ex, ex - 1) - p + 127
    low, high = RANGE[bits, dt]
    e = np.clip(np.where(m == 0, low, e), low, high)
    a = np.abs(np.where(finite[..., None], y, 0)) / np.ldexp(1.0, e - 127)[..., None]
    mids = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mids, a, side="left")             # a tie is at the lower of its two
    tie = (i < len(mids)) & (a == mids[np.minimum(i, len(mids) - 1)])
    i = i + (tie & (i % 2 == 1))
    codes = i + np.where(np.signbit(y) & (i >= 0), 1 << (bits - 1), 0)
    codes = np.where(finite[..., None], codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), np.where(finite, e, 255).astype(np.uint8)


def kv_decode(codes, scales, bits):
    """The values that codes stand for; a NaN block for the scale byte 255."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    half = 1 << (bits - 1)
    grid = GRID4 if bits == 4 else np.append(GRID8, np.nan)
    v = grid[codes % half] * np.where(codes >= half, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


def pack(codes, bits):
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(raw, bits):
    return raw if bits == 8 else np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], -1)


def silu(s):
    return np.where(s < -745, -0.0, s / (1 + np.exp(np.clip(-s, -745, 745))))


def silu_rel(s):
    return (2 * np.abs(s) + 6) * U


def conv(x, weight, bias, state, act):
    """One sequence: x [T, C], weight [C, W], state [W - 1, C].  Returns (out, bound, state)."""
    x, weight, state = (np.asarray(v, np.float64) for v in (x, weight, state))
    W = weight.shape[1]
    line = np.concatenate([state, x])
    s, mag = np.zeros_like(x), np.zeros_like(x)
    if bias is not None:
        s, mag = s + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    for w in range(W):
        s = s + weight[:, w] * line[w:w + len(x)]
        mag = mag + np.abs(weight[:, w] * line[w:w + len(x)])
    err = (W + 1) * U * mag
    if not act:
        return s, err, line[len(x):]
    y = silu(s)
    return y, 1.1 * err + np.abs(y) * silu_rel(s) + 1e-36, line[len(x):]


def scan(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=True, piece=1):
    """One sequence: x, dt, z [T, Di], B, C [T, N], A, state [Di, N].  Returns (out,
    out_bound, state, state_bound)."""
    x, dt, A, B, C = (np.asarray(v, np.float64) for v in (x, dt, A, B, C))
    h = np.array(state, np.float64)
    err = np.zeros_like(h)
    s = dt if dt_bias is None else dt + np.asarray(dt_bias, np.float64)
    if softplus:
        delta = np.maximum(s, 0) + np.log1p(np.exp(-np.abs(s)))
        ed = 1.25 * np.abs(s) * U / (1 + np.exp(np.clip(-s, -700, 700))) + 16 * U * delta
    else:
        delta, ed = s, np.abs(s) * U
    out, bound = np.zeros_like(x), np.zeros_like(x)
    for t in range(len(x)):
        d, e = delta[t][:, None], ed[t][:, None]
        a, u = np.exp(d * A), d * x[t][:, None] * B[t][None]
        rel = np.abs(A) * e + np.abs(d * A) * (3 + piece) * U + 4 * U
        err = a * err + np.abs(a * h) * rel + np.abs(x[t][:, None] * B[t][None]) * e + 3 * U * np.abs(u) + 2.0 ** -126
        h = a * h + u
        y, mag, ye = h @ C[t], np.abs(h) @ np.abs(C[t]), err @ np.abs(C[t])
        if D is not None:
            y, mag = y + np.asarray(D, np.float64) * x[t], mag + np.abs(np.asarray(D, np.float64) * x[t])
        ye = ye + (A.shape[1] + 4) * U * mag
        if z is not None:
            g = silu(np.asarray(z[t], np.float64))
            y, ye = y * g, ye * np.abs(g) + np.abs(y * g) * (silu_rel(np.asarray(z[t], np.float64)) + U) + 1e-36
        out[t], bound[t] = y, ye
    return out, bound, h, err
