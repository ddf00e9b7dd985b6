"""Attention of a decode batch over a shared prefix and paged suffixes, against
the 64-bit oracle: head layouts, types, page sizes, empty and ragged suffixes,
no prefix, garbage past the lengths, ids outside the pages, strided operands,
graph replays.  Tolerances are the oracle's bounds plus the output's rounding."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gemm_decode_q1_amd as Q

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    Q.load_library()
    assert Q.q1_device_supported(0), Q.q1_last_error()
    yield
    torch.cuda.synchronize()


def npd(t):
    return t.detach().double().cpu().numpy()


def draw(seed, B, Hq, Hkv, D, P, lens, page, dt, garbage=True):
    """Operands; pages beyond a length hold NaN (rows that must not be used)."""
    r = np.random.default_rng(seed)
    most = max(lens) if lens else 0
    per = max(1, -(-most // page))
    t = lambda *s: torch.from_numpy(r.standard_normal(s)).to(DT[dt]).cuda()  # noqa: E731
    q = 2.0 * t(B, Hq, D)
    kp, vp = t(P, Hkv, D), t(P, Hkv, D)
    pages = B * per + 3
    kc, vc = t(pages, page, Hkv, D), t(pages, page, Hkv, D)
    table = r.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    if garbage:
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            for i in range(n):
                used[table[b, i // page], i % page] = True
        bad = torch.from_numpy(~used).cuda()
        kc[bad] = float("nan")
        vc[bad] = float("nan")
    return q, kp, vp, kc, vc, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def rows(x, table, n, page):
    t = table.cpu().numpy()
    flat = npd(x)
    return np.stack([flat[t[i // page], i % page] for i in range(n)]) if n else np.zeros((0, *flat.shape[2:]))


def check(out, lse, q, kp, vp, kc, vc, table, lens, page, out_dt, scale, what, left_out=()):
    pk, pv = npd(kp), npd(vp)
    for b, n in enumerate(lens):
        keys = np.concatenate([pk, rows(kc, table[b], n, page)])
        values = np.concatenate([pv, rows(vc, table[b], n, page)])
        ref, bound, l, lb = R.prefix_attention(npd(q[b]), keys, values, scale)
        eo = np.abs(npd(out[b]) - ref) - bound - R.half_ulp(np.abs(ref) + bound, out_dt)
        print(f"{what} sequence {b} ({n} of its own): out over bound {eo.max():.3g}", flush=True)
        assert np.isfinite(npd(out[b])).all() and eo.max() <= 0
        el = npd(lse[b])
        if keys.shape[0] == 0:
            assert (el == -np.inf).all() and (npd(out[b]) == 0).all()
        else:
            assert (np.abs(el - l) <= lb).all()


@pytest.mark.parametrize("B,Hq,Hkv,D,P,lens,page,dt,out_dt", [
    (1, 1, 1, 64, 1, [0], 16, "bf16", "f32"),
    (1, 8, 8, 128, 1, [1], 1, "f16", "f32"),
    (4, 24, 4, 128, 519, [40, 0, 17, 1], 16, "bf16", "bf16"),
    (3, 12, 2, 256, 300, [100, 33, 64], 17, "bf16", "f32"),
    (5, 8, 1, 64, 1000, [5, 300, 0, 129, 128], 48, "f16", "f16"),
    (2, 6, 6, 128, 0, [70, 257], 64, "bf16", "f32"),
    (17, 6, 2, 64, 130, [3 * i for i in range(17)], 16, "f16", "f32"),
    (40, 4, 1, 128, 65, [(7 * i) % 50 for i in range(40)], 32, "bf16", "f32"),
    (2, 32, 1, 256, 90, [31, 32], 16, "f16", "f32"),
    (2, 40, 1, 64, 77, [200, 3], 100, "bf16", "f32"),
    (1, 4, 2, 128, 6000, [2000], 64, "bf16", "f32"),
])
def test_against_oracle(B, Hq, Hkv, D, P, lens, page, dt, out_dt):
    ops = draw(B + P, B, Hq, Hkv, D, P, lens, page, dt)
    if P == 0:
        out, lse = Q.q1_prefix_attn(ops[0], None, None, *ops[3:], out_dtype=DT[out_dt])
    else:
        out, lse = Q.q1_prefix_attn(*ops, out_dtype=DT[out_dt])
    check(out, lse, *ops[:6], lens, page, out_dt, D ** -0.5, f"B={B} Hq={Hq}/{Hkv} D={D} P={P}")


def test_prefix_alone():
    q, kp, vp, *_ = draw(1, 3, 6, 2, 128, 200, [0, 0, 0], 16, "bf16")
    out, lse = Q.q1_prefix_attn(q, kp, vp, out_dtype=torch.float32)
    for b in range(3):
        ref, bound, l, lb = R.prefix_attention(npd(q[b]), npd(kp), npd(vp), 128 ** -0.5)
        assert (np.abs(npd(out[b]) - ref) <= bound + R.half_ulp(ref, "f32")).all() and (np.abs(npd(lse[b]) - l) <= lb).all()


def test_rows_with_nothing():
    """No prefix and an empty suffix (also a negative length): zeros, lse = -infinity."""
    ops = draw(2, 3, 4, 2, 64, 0, [0, 5, 0], 4, "bf16")
    lens = torch.tensor([0, 5, -3], dtype=torch.int32).cuda()
    out, lse = Q.q1_prefix_attn(ops[0], None, None, *ops[3:6], lens)
    assert (out[[0, 2]] == 0).all() and (lse[[0, 2]] == -float("inf")).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


def test_scores_far_apart():
    """Scores of thousands, equal and opposite: the maximum is taken out before exp."""
    B, Hq, Hkv, D, P, lens, page = 2, 4, 2, 64, 100, [30, 0], 8
    q, kp, vp, kc, vc, table, L = draw(3, B, Hq, Hkv, D, P, lens, page, "bf16")
    q = q * 100
    out, lse = Q.q1_prefix_attn(q, kp, vp, kc, vc, table, L, out_dtype=torch.float32)
    check(out, lse, q, kp, vp, kc, vc, table, lens, page, "f32", D ** -0.5, "large scores")
    out, lse = Q.q1_prefix_attn(q, kp, vp, kc, vc, table, L, scale=0.0, out_dtype=torch.float32)
    check(out, lse, q, kp, vp, kc, vc, table, lens, page, "f32", 0.0, "scale 0")


def test_ids_and_lengths_out_of_range():
    """A page id outside the pages leaves its tokens out; a length is clamped to the table."""
    B, Hq, Hkv, D, P, page = 2, 4, 2, 128, 50, 16
    q, kp, vp, kc, vc, table, _ = draw(4, B, Hq, Hkv, D, P, [48, 48], page, "bf16", garbage=False)
    table[0, 1] = -7
    table[1, 2] = 10 ** 6
    lens = torch.tensor([48, 10 ** 9], dtype=torch.int32).cuda()
    out, lse = Q.q1_prefix_attn(q, kp, vp, kc, vc, table, lens, out_dtype=torch.float32)
    for b, keep in ((0, [0, 2]), (1, [0, 1])):
        ids = table[b][keep].long()
        keys = np.concatenate([npd(kp), npd(kc[ids]).reshape(-1, Hkv, D)])
        values = np.concatenate([npd(vp), npd(vc[ids]).reshape(-1, Hkv, D)])
        ref, bound, l, lb = R.prefix_attention(npd(q[b]), keys, values, D ** -0.5)
        assert (np.abs(npd(out[b]) - ref) <= bound + R.half_ulp(ref, "f32")).all() and (np.abs(npd(lse[b]) - l) <= lb).all()


def test_strided_operands():
    """q as a slice of a projection's rows, the prefix as slices of a fused key/value buffer."""
    B, Hq, Hkv, D, P, lens, page = 3, 6, 2, 64, 90, [10, 0, 33], 16
    q, kp, vp, kc, vc, table, L = draw(5, B, Hq, Hkv, D, P, lens, page, "f16")
    big = torch.cat([q.flatten(1), torch.ones_like(q).flatten(1)], 1)
    qs = big[:, :Hq * D].unflatten(1, (Hq, D))
    kv = torch.stack([kp, vp], 1)
    a = Q.q1_prefix_attn(qs, kv[:, 0], kv[:, 1], kc, vc, table, L)
    b = Q.q1_prefix_attn(q, kp, vp, kc, vc, table, L)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_stream_and_bits():
    B, Hq, Hkv, D, P, lens, page = 4, 24, 4, 128, 3001, [40, 0, 500, 1], 16
    ops = draw(6, B, Hq, Hkv, D, P, lens, page, "bf16")
    want = [x.clone() for x in Q.q1_prefix_attn(*ops)]
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(Q.q1_prefix_attn(*ops), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = Q.q1_prefix_attn(*ops)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = Q.q1_prefix_attn(*ops)
    for i in range(4):
        got[0].zero_()
        got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        Q.q1_prefix_attn(ops[0] * i, *ops[1:])


@pytest.mark.parametrize("what", ["dtype", "pages", "table", "nothing", "host", "half"])
def test_binding_refusals(what):
    q, kp, vp, kc, vc, table, L = draw(7, 2, 4, 2, 64, 20, [3, 4], 4, "bf16")
    if what == "dtype":
        kp = kp.half()
    elif what == "pages":
        kc = kc.transpose(1, 2)
    elif what == "table":
        table = table.long()
    elif what == "nothing":
        kp = vp = kc = vc = table = L = None
    elif what == "host":
        L = L.cpu()
    else:
        vp = None
    with pytest.raises(ValueError):
        Q.q1_prefix_attn(q, kp, vp, kc, vc, table, L)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_offsets_past_32_bits(dt):
    """A cache of over 4 GiB whose last pages are used, and prefix rows so far apart that
    their offsets pass 32 bits."""
    B, Hq, Hkv, D, page, pages, P = 2, 8, 4, 128, 64, 70000, 9000
    lens = [130, 65]
    q, kp, vp, kc, vc, table, n = draw(77, B, Hq, Hkv, D, P, lens, page, dt)
    far = pages - kc.shape[0]
    big = [torch.empty(pages, page, Hkv, D, dtype=DT[dt], device="cuda") for _ in range(2)]
    for b, small in zip(big, (kc, vc)):
        b[far:] = small
    ld = 1 << 18
    wide = [torch.empty(P * ld, dtype=DT[dt], device="cuda").as_strided((P, Hkv, D), (ld, D, 1)) for _ in range(2)]
    for w, small in zip(wide, (kp, vp)):
        w.copy_(small)
    want = Q.q1_prefix_attn(q, kp, vp, kc, vc, table, n, out_dtype=torch.float32)
    got = Q.q1_prefix_attn(q, wide[0], wide[1], big[0], big[1], table + far, n, out_dtype=torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(got[0], got[1], q, kp, vp, kc, vc, table, lens, page, "f32", D ** -0.5, "far")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("B,Hq,Hkv,D,P", [(3, 6, 2, 64, 700), (3, 4, 2, 256, 90), (24, 8, 2, 128, 300), (3, 8, 2, 128, 0)])
def test_nan_and_infinity_in_what_counts(B, Hq, Hkv, D, P, dt):
    """A NaN or an infinite score makes its rows NaN, the sum of weights too (-infinity would say that there is
    no token); a NaN or infinite value its column, not the sum; other rows and columns keep their bits."""
    lens, page, group = [9 + 5 * (b % 7) for b in range(B)], 16, Hq // Hkv
    q, kp, vp, kc, vc, table, n = draw(21, B, Hq, Hkv, D, P, lens, page, dt)
    call = lambda q, kp, vp, kc, vc: Q.q1_prefix_attn(q, *((kp, vp) if P else (None, None)), kc, vc, table, n,  # noqa: E731
                                                      out_dtype=torch.float32)
    clean, clean_lse = call(q, kp, vp, kc, vc)
    nan, inf = float("nan"), float("inf")
    where = (table[1, 0].item(), 3)  # a token of sequence 1 that counts

    def same_but(got, rows, columns, lse_too):
        """NaN (for a bad value: or infinite) in `rows` (sequence, head) and `columns`, the clean run's bits elsewhere."""
        out, lse = got
        hit = torch.zeros(B, Hq, D, dtype=torch.bool).cuda()
        for b, h in rows:
            hit[b, h, columns] = True
        assert (out[hit].isnan() if lse_too else ~out[hit].isfinite()).all() and torch.equal(out[~hit], clean[~hit])
        hit = hit.any(-1) if lse_too else torch.zeros_like(lse, dtype=torch.bool)
        assert lse[hit].isnan().all() and torch.equal(lse[~hit], clean_lse[~hit])

    every = slice(None)
    x = q.clone()
    x[1, 2, 7] = nan
    same_but(call(x, kp, vp, kc, vc), [(1, 2)], every, True)
    first = [(1, h) for h in range(group)]  # the rows of key head 0
    x = kc.clone()
    x[where[0], where[1], 0, 5] = nan
    same_but(call(q, kp, vp, x, vc), first, every, True)
    x[where[0], where[1], 0] = 0
    x[where[0], where[1], 0, 5] = inf
    y = q.clone()
    y[1, :, 5] = 1.0  # a score of +infinity
    out, lse = call(y, kp, vp, x, vc)
    assert out[1, :group].isnan().all() and lse[1, :group].isnan().all()
    assert torch.isfinite(out[:, group:]).all() and torch.isfinite(lse[:, group:]).all() and torch.isfinite(out[2:]).all()
    for bad in (nan, inf, -inf):
        x = vc.clone()
        x[where[0], where[1], 0, 5] = bad
        same_but(call(q, kp, vp, kc, x), first, [5], False)
    if P:
        x = kp.clone()
        x[P - 1, 1, 0] = nan
        same_but(call(q, x, vp, kc, vc), [(b, h) for b in range(B) for h in range(group, Hq)], every, True)
