"""The chunked gated delta rule in NumPy's fp32, with its fp32 operands as a number of
bf16 parts, and the recurrence in fp32: what precision either form reaches.  One head,
keys and queries normalised; shares no code with the HIP path."""
import numpy as np

F = np.float32


def cut(x):
    """The leading 8 significant bits."""
    return (np.ascontiguousarray(x, F).view(np.uint32) & 0xffff0000).view(F)


def nearest(x):
    """Rounded to the nearest bf16."""
    u = np.ascontiguousarray(x, F).view(np.uint32)
    return ((u + 0x7fff + (u >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(F)


def parts(x, n):
    got, x = [], np.asarray(x, F)
    for _ in range(n):
        got.append(cut(x))
        x = (x - got[-1]).astype(F)
    return got


def product(a, b, most):
    """Sum of the products of parts i of a and j of b with i + j <= most, small ones first."""
    s = 0
    for d in range(most, -1, -1):
        for i in range(len(a)):
            if 0 <= d - i < len(b):
                s = (s + (a[i] @ b[d - i]).astype(F)).astype(F)
    return s


def norms(x):
    return (1 / np.sqrt((x * x).sum(-1) + F(1e-6))).astype(F)


def chunked(q, k, v, g, beta, S, scale, state_parts=3, out_parts=3, C=64):
    q, k, v, g, beta, S = (np.asarray(x, F) for x in (q, k, v, g, beta, S))
    out, scale = np.zeros(v.shape, F), F(scale)
    rk, rq = norms(k), norms(q)
    n, m = state_parts, out_parts
    for t in range(0, len(q), C):
        s = slice(t, min(len(q), t + C))
        G = np.cumsum(g[s].astype(np.float64))
        D = np.exp(np.tril(G[:, None] - G[None])).astype(F)
        A = np.tril(beta[s][:, None] * rk[s][:, None] * rk[s][None] * (k[s] @ k[s].T) * D, -1)
        P = np.tril(scale * rq[s][:, None] * rk[s][None] * (q[s] @ k[s].T) * D)
        T = np.linalg.inv(np.eye(len(G)) + A.astype(np.float64)).astype(F) * beta[s][None]
        eG, left = np.exp(G).astype(F), np.exp(G[-1] - G).astype(F)
        R = (v[s] - (rk[s] * eG)[:, None] * product([k[s]], parts(S, n), n - 1)).astype(F)
        V = product(parts(T, n), parts(R, n), n - 1)
        out[s] = (scale * rq[s] * eG)[:, None] * product([q[s]], parts(S, m), m - 1) + product(parts(P, m), parts(V, m), m - 1)
        S = (eG[-1] * S + product([k[s].T], parts((rk[s] * left)[:, None] * V, n), n - 1)).astype(F)
    return out, S


def recurrent(q, k, v, g, beta, S, scale):
    q, k, v, g, beta, S = (np.asarray(x, F) for x in (q, k, v, g, beta, S))
    out, rk, rq = np.zeros(v.shape, F), norms(k), norms(q)
    for t in range(len(q)):
        a = np.exp(g[t])
        d = (beta[t] * (v[t] - a * (rk[t] * (k[t] @ S)))).astype(F)
        out[t] = F(scale) * (a * (rq[t] * (q[t] @ S)) + (q[t] @ k[t]) * rk[t] * rq[t] * d)
        S = ((k[t] * rk[t])[:, None] * d[None] + a * S).astype(F)
    return out, S


def error(got, exact):
    """Relative error in the Euclidean norm."""
    return np.linalg.norm(np.asarray(got, np.float64) - exact) / np.linalg.norm(exact)


# The chunked form rounds the state once a chunk where the recurrence does it every token, and has sums of
# the same number of terms: in fp32 it is no worse.  A factor of two allows for another order of its sums,
# and one of two for matrix cores that cut off where they add.  One part too few leaves out 2^-16 of a
# value, more than eight times the recurrence's error.
LIMIT = 4.0

# Log decays a token (scaled): states that last, so that what a chunk loses adds up.
RATES = (0.0, 1e-3, 0.1)
