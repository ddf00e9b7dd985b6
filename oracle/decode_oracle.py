"""CPU oracle of the decode-step operators: NumPy, 64 bits, straight from the
definitions in ``include/q1_decode.h``.  Shares no code with the HIP path.

Error bounds beside the values:

* ``delta_rule``: every token's update is, per column s of the state, the map
  s -> a (I - beta k k^T) s + beta v k, which for |k| <= 1, 0 <= beta <= 1 and
  a <= 1 does not lengthen a difference.  So an error e(t) of a column obeys
  e(t) <= a e(t-1) + c 2^-24 (|s| + |beta v|), with c 2^-24 the relative error
  of one token's fp32 arithmetic; the output adds scale |q| (e + c 2^-24 |s|).
  A dot product of n fp32 terms is off by at most n 2^-24 of the sum of the
  absolute terms, itself at most the product of the norms; a token has two of
  Dk terms and a handful of single roundings: c = 2 Dk + 16.  The chunked form
  chains a product with the state (Dk terms), one with the chunk's inverse (64
  terms), one with the chunk's keys or scores (64 terms) and makes the inverse
  from scores of Dk terms; with row sums of the inverse's absolute values of
  at most 4, c = 4 (2 Dk + 128) + 16.
* ``prefix_attention``: a score is off by at most ds = (D + 4) 2^-24 scale
  sum |q k|; weights by a factor within 2 ds + 2^-20; the weighted sum of n
  terms by (n + 8) 2^-24; weights enter the second product as a pair of 8-bit
  significands (2^-16): with A = sum p |v|, the output is off by at most
  A (2 ds + 2^-20 + (n + 8) 2^-24 + 2^-16).
* ``sample`` gives the token; ``sample_choices`` also those that weights within
  the exponential's error of the exact ones would give.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24


def delta_rule(q, k, v, g, beta, state, l2norm, scale, c):
    """One sequence: q, k [T, Hk, Dk], v [T, Hv, Dv], g, beta [T, Hv], state
    [Hv, Dk, Dv].  Returns (out, out_bound, state, state_bound)."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    S = np.array(state, np.float64)
    rep = v.shape[1] // k.shape[1]
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    err = np.zeros((S.shape[0], S.shape[2]))
    out, bound = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(q.shape[0]):
        qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
        a = np.exp(g[t])[:, None]
        before = np.sqrt((S * S).sum(1))
        S = a[:, :, None] * S
        pred = np.einsum("hkv,hk->hv", S, kt)
        S = S + kt[:, :, None] * (beta[t][:, None] * (v[t] - pred))[:, None, :]
        err = a * err + c * EPS * (before + np.abs(beta[t][:, None] * v[t]))
        out[t] = scale * np.einsum("hkv,hk->hv", S, qt)
        size = np.sqrt((qt * qt).sum(-1))[:, None]
        bound[t] = abs(scale) * size * (err + c * EPS * np.maximum(before, np.sqrt((S * S).sum(1))))
    return out, bound, S, np.broadcast_to(err[:, None, :], S.shape)


def prefix_attention(q, keys, values, scale):
    """One sequence: q [Hq, D], keys and values [n, Hkv, D].  Returns (out, bound, lse, lse_bound)."""
    q, keys, values = (np.asarray(x, np.float64) for x in (q, keys, values))
    hq, d = q.shape
    n, hkv = keys.shape[0], keys.shape[1]
    if n == 0:
        return np.zeros((hq, d)), np.zeros((hq, d)), np.full(hq, -np.inf), np.zeros(hq)
    head = np.arange(hq) // (hq // hkv)
    s = scale * np.einsum("hd,nhd->hn", q, keys[:, head])
    ds = (d + 4) * EPS * abs(scale) * np.einsum("hd,nhd->hn", np.abs(q), np.abs(keys[:, head])).max(1)
    m = s.max(1)
    p = np.exp(s - m[:, None])
    total = p.sum(1)
    p = p / total[:, None]
    out = np.einsum("hn,nhd->hd", p, values[:, head])
    A = np.einsum("hn,nhd->hd", p, np.abs(values[:, head]))
    rel = 2 * ds + 2.0 ** -20 + (n + 8) * EPS + 2.0 ** -16
    lse = m + np.log(total)
    return out, A * rel[:, None], lse, ds + 2.0 ** -20 + (n + 8) * EPS + 4 * EPS * np.abs(lse)


def half_ulp(x, dtype):
    """Half the spacing of the output type at |x|."""
    bits, low = {"f32": (23, -126), "f16": (10, -14), "bf16": (7, -126)}[dtype]
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** low)))
    return 0.5 * 2.0 ** (np.maximum(e, low) - bits)


NEAR = 2.0 ** -22  # a 32-bit exponential is within two units in the last place


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of float32 logits: (token, logprob) by the definition."""
    return sample_choices(row, u, temperature, top_k, top_p, min_p, 0.0)[0]


def sample_choices(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, near=NEAR):
    """The (token, logprob) by the definition, then those it gives for weights
    within `near` of these: the draw, the top-p cut and the min-p cut each moved
    by that much of the weights that are not exact (a largest logit's is)."""
    x = np.asarray(row, np.float32).copy()
    x[np.isnan(x)] = -np.inf
    top = x.max()
    if top == -np.inf:
        return [(-1, -np.inf)]
    T = np.float32(temperature)
    greedy = not T > 0
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        d = np.where(x == top, np.float32(0), x - top).astype(np.float32)
        if not greedy:
            d = (d / T).astype(np.float32)
        e = np.exp(d.astype(np.float64)).astype(np.float32)
    w = np.floor(e.astype(np.float64) * 2.0 ** 40).astype(np.int64)
    order = np.lexsort((np.arange(len(x)), -x))[:1 if greedy else (top_k if top_k > 0 else len(x))]
    order = order[(w[order] > 0)]
    total = lambda at: int(w[at].sum())                 # noqa: E731
    loose = lambda at: near * int(w[at][e[at] < 1].sum())  # noqa: E731
    before = np.cumsum(w[order]) - w[order]
    cuts = [order]
    if top_p < 1:
        W, move = total(order), loose(order)
        bound = max(1, int(float(np.float32(top_p)) * float(W)))
        cuts = [order[before < max(1, bound + s)] for s in (0, -move, move)]
    mp = np.float32(min(min_p, 1.0)) if min_p > 0 else np.float32(0)
    found = []
    for i, cut in enumerate(cuts):
        for s in (0.0, -near, near):
            kept = np.sort(cut[~(e[cut].astype(np.float64) * (1 + s * (e[cut] < 1)) < mp)])
            W, move = total(kept), loose(kept)
            r = min(int(float(np.float32(min(u, 1.0))) * float(W)), W - 1) if u > 0 else 0
            upto = np.cumsum(w[kept])
            mine = int(np.searchsorted(upto, r, side="right"))
            lo = int(np.searchsorted(upto, r - move, side="right"))
            hi = min(int(np.searchsorted(upto, r + move, side="right")), len(kept) - 1)
            for j in [mine, *range(lo, hi + 1)]:
                c = (int(kept[j]), float(np.log(w[kept[j]] / W)))
                if c not in found:
                    found.append(c)
    return found
