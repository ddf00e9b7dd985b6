"""What a decoder remembers between tokens, as measured cases.

Four operators: keys and values quantised to 4 or 8 bits as they are written to
pages, and read back (``q1_kv_write``, ``q1_kv_read``); attention over such pages
(``q1_kv_attn``); the short causal convolution (``q1_conv_step``,
``q1_conv_prefill``); the selective state space scan (``q1_scan_step``,
``q1_scan_prefill``).  ``run`` computes them in plain torch operations in 32 bits,
or, where ``own`` is true, through this repository's package.

Keys and values in pages: blocks of 32 consecutive elements of a (token, head)
share a scale 2^e, e the smallest integer with max |x| <= 1.75 * 2^(e + p), held as
the byte e + 127.  With 4 bits p = 2 and an element is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
a sign (E2M1); with 8 bits p = 8 and it is E4M3, largest 448.  Nearest, ties to even.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_BLOCK = 32
_TOP = {4: 2, 8: 8}                                       # p
_LOW = {4: 2, 8: 10}                                      # scale bytes whose every value is a normal bf16
_HIGH = {(4, "bf16"): 252, (8, "bf16"): 246, (4, "f16"): 140, (8, "f16"): 134}  # and finite in the operands' type


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # a decode step of eight sequences: their new rows, in 4 bits, where latency counts
        dict(name="cache one step", op="cache", tokens=8, Hkv=4, D=256, bits=4, page=64, dt="bf16"),
        # a ragged batch's prompts in 8 bits
        dict(name="cache prompts 8 bits", op="cache", tokens=4099, Hkv=2, D=64, bits=8, page=17, dt="f16"),
        # one long prompt in 4 bits
        dict(name="cache long prompt", op="cache", tokens=16384, Hkv=8, D=128, bits=4, page=16, dt="bf16"),
        # a few users with short contexts
        dict(name="attn short", op="attn", B=4, T=1, Hkv=4, group=6, D=128, most=519, page=16, bits=4, dt="bf16"),
        # a batch of answers to documents, some of them just begun
        dict(name="attn batch", op="attn", B=32, T=1, Hkv=4, group=6, D=256, most=8201, page=64, bits=4, dt="bf16"),
        # eight users of very long contexts, three drafted tokens each
        dict(name="attn long drafted", op="attn", B=8, T=3, Hkv=8, group=4, D=128, most=65537, page=48, bits=4, dt="f16"),
        # the last thousand tokens of two prompts over all that came before, in 8 bits
        dict(name="attn prompt 8 bits", op="attn", B=2, T=1000, Hkv=4, group=6, D=128, most=5003, page=64, bits=8, dt="bf16"),
        # eight sequences' next tokens: keys, queries and values of the delta rule's 16 + 16 + 48 heads of 128
        dict(name="conv step", op="conv step", B=8, T=1, C=10240, W=4, dt="bf16", bias=False),
        # a ragged batch of prompts through the same
        dict(name="conv prompts", op="conv", tokens=16384, nseq=5, C=10240, W=4, dt="bf16", bias=True),
        # one user's next token, where latency counts
        dict(name="scan step", op="scan step", B=1, T=1, Di=5120, N=16, dt="bf16", dt32=False),
        # a ragged batch of prompts, single tokens among them
        dict(name="scan prompts", op="scan", tokens=4099, nseq=7, Di=5120, N=16, dt="f16", dt32=True),
        # one long prompt
        dict(name="scan long prompt", op="scan", tokens=16384, nseq=1, Di=5120, N=16, dt="bf16", dt32=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["cache", "attn", "attn", "conv step", "conv", "scan step", "scan"])
    dt = rng.choice(["bf16", "f16"])
    if op == "cache":
        c = dict(op=op, tokens=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128, 256]),
                 bits=rng.choice([4, 4, 8]), page=rng.choice([1, 16, 17, 48, 64]), dt=dt)
        while c["tokens"] * c["Hkv"] * c["D"] > 16384 * 8 * 128:
            c["tokens"] = c["tokens"] // 2 + 1
        return c
    if op == "attn":
        c = dict(op=op, B=_log(rng, 1, 48), T=rng.choice([1, 1, 1, 2, 5, 64, 301]), Hkv=rng.choice([1, 2, 4, 8]),
                 group=rng.choice([1, 3, 4, 6, 8]), D=rng.choice([64, 128, 256]), most=_log(rng, 1, 65536),
                 page=rng.choice([1, 16, 17, 48, 64]), bits=rng.choice([4, 4, 8]), dt=dt)
        while (c["B"] * c["Hkv"] * c["D"] * c["most"] > 8 * 8 * 128 * 32000
               or c["B"] * c["T"] * c["Hkv"] * c["group"] * c["D"] * c["most"] > 2 * 1000 * 24 * 128 * 2500):
            c["most"] = c["most"] // 2 + 1
            c["B"] = c["B"] // 2 + 1
            c["T"] = c["T"] // 2 + 1
        return c
    if op in ("conv step", "conv"):
        c = dict(op=op, C=8 * _log(rng, 8, 1280), W=rng.choice([2, 3, 4, 4, 4]), dt=dt, bias=rng.random() < 0.5)
        if op == "conv step":
            return dict(c, B=_log(rng, 1, 128), T=rng.choice([1, 1, 1, 2, 4]))
        return dict(c, tokens=_log(rng, 1, 16000), nseq=_log(rng, 1, 16))
    c = dict(op=op, Di=8 * _log(rng, 8, 640), N=rng.choice([8, 16, 16, 16, 32]), dt=dt, dt32=rng.random() < 0.3)
    if op == "scan step":
        return dict(c, B=_log(rng, 1, 128), T=rng.choice([1, 1, 1, 2, 4]))
    return dict(c, tokens=_log(rng, 1, 8000), nseq=_log(rng, 1, 16))


def _lengths(case):
    """Lengths of a ragged batch: from the case alone, so that its work is known."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "attn":
        got = [max(1, int(case["most"] * r.random() ** 0.7)) for _ in range(case["B"])]
        got[r.randrange(len(got))] = case["most"]
        return got
    cuts = sorted(r.randint(0, case["tokens"]) for _ in range(case["nseq"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]


# --- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _pages(pages, case):
    """Empty pages: codes and scale bytes of keys and values."""
    lead = (pages, case["Hkv"], case["page"])
    zero = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    return dict(k=zero(*lead, case["D"] * case["bits"] // 8), v=zero(*lead, case["D"] * case["bits"] // 8),
                k_scales=zero(*lead, case["D"] // _BLOCK), v_scales=zero(*lead, case["D"] // _BLOCK))


def _handle(st, case):
    """The framework's handle of the pages, which a program keeps."""
    st["bits"], st["dt"] = case["bits"], case["dt"]
    if own:
        import gemm_decode_q1_amd as Q
        st["cache"] = Q.PackedKV(st["k"], st["v"], st["k_scales"], st["v_scales"], case["bits"])
    return st


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "cache":
        n, hkv, d = case["tokens"], case["Hkv"], case["D"]
        pages = -(-n // case["page"]) + 3
        # keys have a few large channels; both are slices of one projection's rows
        wide = 1 + 6 * (_rand(g, hkv, d) < 0.04)
        x = torch.cat([(_randn(g, n, hkv, d) * wide).flatten(1), _randn(g, n, hkv * d)], 1).to(_DT[case["dt"]])
        x = x.view(n, 2, hkv, d)
        slots = torch.randperm(pages * case["page"], device="cuda", generator=g)[:n].to(torch.int32)
        return _handle(dict(_pages(pages, case), op=op, new_k=x[:, 0], new_v=x[:, 1], slots=slots), case)
    if op == "attn":
        b, t, hkv, d, page = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
        lens = _lengths(case)
        per = -(-case["most"] // page)
        pages = sum(-(-n // page) for n in lens) + 2
        st = dict(_pages(pages, case), op=op, q=(1.5 * _randn(g, b, t, hkv * case["group"], d)).to(_DT[case["dt"]]))
        step = max(1, (1 << 26) // (hkv * page * d))
        for name in ("k", "v"):
            for i in range(0, pages, step):
                n = min(step, pages - i)
                codes, scale = _quantise(_randn(g, n, hkv, page, d).to(_DT[case["dt"]]), case["bits"], case["dt"])
                st[name][i:i + n], st[name + "_scales"][i:i + n] = _pack(codes, case["bits"]), scale
        ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        table, at = torch.zeros(b, per, dtype=torch.int32, device="cuda"), 0
        for i, n in enumerate(lens):
            k = -(-n // page)
            table[i, :k] = ids[at:at + k]
            at += k
        st["table"], st["lens"] = table, torch.tensor(lens, dtype=torch.int32).cuda()
        return _handle(st, case)
    step = op.endswith("step")
    n = case["B"] if step else case["nseq"]
    lead = (case["B"], case["T"]) if step else (case["tokens"],)
    dt, pool = _DT[case["dt"]], n + 3
    st = dict(op=op, slots=torch.randperm(pool, device="cuda", generator=g)[:n].to(torch.int32))
    if not step:
        st["lens"] = _lengths(case)
        st["cu"] = torch.tensor([0] + list(np.cumsum(st["lens"])), dtype=torch.int32).cuda()
    if op.startswith("conv"):
        c, w = case["C"], case["W"]
        st["x"] = _randn(g, *lead, c).to(dt)
        st["weight"] = (_randn(g, c, w) * w ** -0.5).to(dt)
        st["bias"] = (0.3 * _randn(g, c)).to(dt) if case["bias"] else None
        st["state"] = _randn(g, pool, w - 1, c).to(dt)
        return st
    di, ns = case["Di"], case["N"]
    x = _randn(g, *lead, 2 * di + 2 * ns).to(dt)  # one row of a projection: x, gate, B, C
    st["x"], st["z"] = x[..., :di], x[..., di:2 * di]
    st["Bt"], st["Ct"] = x[..., 2 * di:2 * di + ns], x[..., 2 * di + ns:]
    st["dt"] = 0.7 * _randn(g, *lead, di)
    if not case["dt32"]:
        st["dt"] = st["dt"].to(dt)
    # steps of 0.001 to 0.1 and rates of 1 to N, each off by a little
    first = torch.exp(_rand(g, di) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = first + torch.log(-torch.expm1(-first))
    st["A"] = -torch.arange(1, ns + 1, device="cuda") * torch.exp(0.1 * _randn(g, di, ns))
    st["D"] = 1 + 0.1 * _randn(g, di)
    st["state"] = _randn(g, pool, di, ns)
    return st


# --- plain forms ------------------------------------------------------------

def _quantise(x, bits, dt):
    """Codes (sign and magnitude as whole numbers of the format) and scale bytes of blocks."""
    y = x.float().unflatten(-1, (-1, _BLOCK))
    top = y.abs().amax(-1)
    e = ((top.view(torch.int32) + 0x1fffff) >> 23) - _TOP[bits]
    e = e.clamp(_LOW[bits], _HIGH[bits, dt])
    y = (y / (e << 23).view(torch.float32)[..., None]).flatten(-2)
    a = y.abs()
    if bits == 4:
        a = a.clamp(max=6.0)
        low, mid = torch.round(2 * a), torch.round(a)
        code = torch.where(a < 2, low, torch.where(a < 4, mid + 2, torch.round(a / 2) + 4))
        code = code.to(torch.uint8)
        return code | ((y < 0).to(torch.uint8) << 3), e.to(torch.uint8)
    a = a.clamp(max=448.0)
    ex = torch.clamp((a.view(torch.int32) >> 23) - 127, min=-6)      # exponent of the step, times 8
    unit = ((ex + 124) << 23).view(torch.float32)
    m = torch.round(a / unit).to(torch.int32)                        # 0..16, a power of two at the top
    code = torch.where(m == 0, 0, m + ((ex + 6) << 3))               # 8..15 of exponent ex: field ex + 7, less the 8 in m
    return code.to(torch.uint8) | ((y < 0).to(torch.uint8) << 7), e.to(torch.uint8)


def _pack(codes, bits):
    """Two 4-bit codes a byte, the even element in the low half."""
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(codes, scales, bits):
    """What stored codes stand for, in 32 bits."""
    if bits == 4:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        m = (c & 7).float()
        a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
        sign = (c >> 3).float()
    else:
        ex, m = ((codes >> 3) & 15).to(torch.int32), (codes & 7).float()
        a = torch.where(ex == 0, m, m + 8) * ((torch.clamp(ex, min=1) + 117) << 23).view(torch.float32)
        sign = (codes >> 7).float()
    s = (scales.to(torch.int32) << 23).view(torch.float32).repeat_interleave(_BLOCK, -1)
    return a * (1 - 2 * sign) * s


def _plain_cache(st):
    page = st["k"].shape[2]
    at = st["slots"].long()
    at, row = at // page, at % page
    out = {}
    for name, x in (("k", st["new_k"]), ("v", st["new_v"])):
        codes, scales = _quantise(x, st["bits"], st["dt"])
        st[name][at, :, row], st[name + "_scales"][at, :, row] = _pack(codes, st["bits"]), scales
        back = _values(st[name][at, :, row], st[name + "_scales"][at, :, row], st["bits"])
        out[name] = back.to(x.dtype)
    return out


def _plain_attn(st):
    q, lens, table = st["q"].float(), st["lens"].long(), st["table"].long()
    b, t, hq, d = q.shape
    hkv, page = st["k"].shape[1], st["k"].shape[2]
    k, v = (_values(st[n][table], st[n + "_scales"][table], st["bits"]).movedim(2, 1).flatten(2, 3) for n in ("k", "v"))
    q = (q.view(b, t, hkv, hq // hkv, d) * d ** -0.5).movedim(1, 2).flatten(2, 3)  # [B, Hkv, T * group, D]
    s = q @ k.transpose(-1, -2)
    seen = lens[:, None] - (t - 1) + torch.arange(t, device="cuda")[None]             # [B, T]
    seen = seen.repeat_interleave(hq // hkv, 1)
    s = s.masked_fill((torch.arange(k.shape[2], device="cuda") >= seen[..., None])[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - base)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, base + total.log())
    back = lambda x: x.unflatten(2, (t, hq // hkv)).movedim(2, 1).flatten(2, 3)  # noqa: E731
    return dict(out=back(o).to(st["q"].dtype), lse=back(lse)[..., 0])


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(st):
    step = st["op"].endswith("step")
    x = st["x"].flatten(0, 1) if step else st["x"]
    slots = st["slots"].long()
    n, keep, c = len(slots), st["state"].shape[1], x.shape[1]
    if step:
        lens = torch.full((n,), st["x"].shape[1], device="cuda")
    else:
        lens = torch.diff(st["cu"]).long()
    first = torch.cumsum(lens, 0) - lens
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), lens, output_size=x.shape[0])
    rows = torch.cat([st["state"][slots].flatten(0, 1), x]).float()
    pos = torch.arange(x.shape[0], device="cuda") - first[seq]

    def at(seq, pos):  # the row of position `pos` of a sequence, negative ones in its state
        return torch.where(pos >= 0, n * keep + first[seq] + pos, seq * keep + keep + pos)

    w = st["weight"].float()
    acc = torch.zeros_like(x, dtype=torch.float32) if st["bias"] is None else st["bias"].float().expand(x.shape).clone()
    for i in range(keep + 1):
        acc += w[:, i] * rows[at(seq, pos - (keep - i))]
    out = _silu(acc).to(x.dtype)
    if keep:
        every = torch.arange(n, device="cuda")[:, None]
        last = at(every, lens[:, None] - keep + torch.arange(keep, device="cuda")[None])
        st["state"][slots] = rows[last.flatten()].view(n, keep, c).to(x.dtype)
    return dict(out=out.view(st["x"].shape), state=st["state"])


def _plain_scan(st):
    """All sequences side by side, a block of tokens' factors at a time; one fused multiply-add a token."""
    step = st["op"].endswith("step")
    slots = st["slots"].long()
    flat = (lambda v: v.flatten(0, 1)) if step else (lambda v: v)  # noqa: E731
    x, z, dt, bt, ct = (flat(st[k]) for k in ("x", "z", "dt", "Bt", "Ct"))
    n = len(slots)
    lens = [st["x"].shape[1]] * n if step else st["lens"]
    length = torch.tensor(lens).cuda()
    first = torch.cumsum(length, 0) - length
    h = st["state"][slots]
    di, ns = h.shape[1:]
    y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    most = max(lens)
    block = max(1, min(256, (1 << 28) // (n * di * ns)))
    for t0 in range(0, most, block):
        pos = torch.arange(t0, min(most, t0 + block), device="cuda")
        inside = pos[:, None] < length[None]                                   # [block, n]
        at = (first[None] + pos[:, None]).clamp(max=x.shape[0] - 1)
        delta = dt[at].float() + st["dt_bias"]
        delta = torch.clamp(delta, min=0) + torch.log1p(torch.exp(-delta.abs()))
        delta = torch.where(inside[..., None], delta, 0.0)
        a = torch.exp(delta[..., None] * st["A"])
        u = (delta * x[at].float())[..., None] * bt[at].float()[:, :, None]
        for t in range(len(pos)):
            h = torch.addcmul(u[t], a[t], h, out=u[t])
        got = (u * ct[at].float()[:, :, None]).sum(-1)
        y[at[inside]] = got[inside]
    y = (y + st["D"] * x.float()) * _silu(z.float())
    st["state"][slots] = h
    return dict(out=y.to(x.dtype).view(st["x"].shape), state=st["state"])


def _plain(st):
    op = st["op"]
    return {"cache": _plain_cache, "attn": _plain_attn}.get(op, _plain_conv if op.startswith("conv") else _plain_scan)(st)


def run(state):
    st = state
    if not own:
        return _plain(st)
    import gemm_decode_q1_amd as Q
    op = st["op"]
    if op == "cache":
        Q.q1_kv_write(st["cache"], st["new_k"], st["new_v"], st["slots"])
        k, v = Q.q1_kv_read(st["cache"], st["slots"], out_dtype=st["new_k"].dtype)
        return dict(k=k, v=v)
    if op == "attn":
        out, lse = Q.q1_kv_attn(st["q"], st["cache"], st["table"], st["lens"])
        return dict(out=out, lse=lse)
    if op == "conv step":
        out = Q.q1_conv_step(st["x"], st["weight"], st["state"], bias=st["bias"], slots=st["slots"])
    elif op == "conv":
        out = Q.q1_conv_prefill(st["x"], st["weight"], st["state"], st["cu"], bias=st["bias"], slots=st["slots"])
    elif op == "scan step":
        out = Q.q1_scan_step(st["x"], st["dt"], st["A"], st["Bt"], st["Ct"], st["state"], D=st["D"], z=st["z"],
                             dt_bias=st["dt_bias"], slots=st["slots"])
    else:
        out = Q.q1_scan_prefill(st["x"], st["dt"], st["A"], st["Bt"], st["Ct"], st["state"], st["cu"], D=st["D"],
                                z=st["z"], dt_bias=st["dt_bias"], slots=st["slots"])
    return dict(out=out, state=st["state"])


# --- the same from the definitions, in 64 bits --------------------------------

def _grid(bits):
    """The magnitudes of the format, in the order of their codes."""
    if bits == 4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    g = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(g[:-1], dtype=torch.float64, device="cuda")


def _exact_round_trip(x, bits, dt):
    y = x.double().unflatten(-1, (-1, _BLOCK))
    m, ex = torch.frexp(y.abs().amax(-1, keepdim=True))        # m in [0.5, 1)
    e = torch.where(2 * m > 1.75, ex, ex - 1) - _TOP[bits]
    e = torch.where(m == 0, -127, e).clamp(_LOW[bits] - 127, _HIGH[bits, dt] - 127)
    scale = ((e.long() + 1023) << 52).view(torch.float64)      # 2^e, bit for bit
    grid = _grid(bits)
    mids = (grid[1:] + grid[:-1]) / 2
    a = (y / scale).abs()
    i = torch.bucketize(a, mids)                               # a tie is at the lower of its two
    up = (i < len(mids)) & (a == mids[i.clamp(max=len(mids) - 1)]) & (i % 2 == 1)
    return (grid[i + up.long()] * scale * torch.where(y < 0, -1.0, 1.0)).flatten(-2)


def _exact_attn(case, st):
    b, t, hq, d = st["q"].shape
    hkv, grp = case["Hkv"], case["group"]
    grid = _grid(case["bits"])
    outs, lses = [], []
    for i, n in enumerate(_lengths(case)):
        ids = st["table"][i, :-(-n // case["page"])].long()

        def rows(name):
            c = st[name][ids].movedim(1, 0).flatten(1, 2)[:, :n]
            if case["bits"] == 4:
                c = torch.stack([c % 16, c // 16], -1).flatten(-2)
            half = 1 << (case["bits"] - 1)
            val = grid[(c % half).long()] * torch.where(c >= half, -1.0, 1.0)
            s = st[name + "_scales"][ids].movedim(1, 0).flatten(1, 2)[:, :n]
            return (val.unflatten(-1, (-1, _BLOCK)) * torch.exp2(s.double() - 127)[..., None]).flatten(-2)

        k, v = rows("k"), rows("v")                            # [Hkv, n, D]
        at = torch.arange(n, device="cuda")
        o, l = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(t, hq, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            q = st["q"][i, :, h * grp:(h + 1) * grp].double()
            s = (q.reshape(-1, d) @ k[h].t().contiguous() / math.sqrt(d)).view(t, grp, n)
            hide = at[None] > n - t + torch.arange(t, device="cuda")[:, None]
            s = s.masked_fill(hide[:, None], -math.inf)
            lse = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
            o[:, h * grp:(h + 1) * grp] = (w.reshape(-1, n) @ v[h]).view(t, grp, d)
            l[:, h * grp:(h + 1) * grp] = lse
        outs.append(o)
        lses.append(l)
    return dict(out=torch.stack(outs), lse=torch.stack(lses))


def _sequences(case):
    lens = [case["T"]] * case["B"] if case["op"].endswith("step") else _lengths(case)
    return [(sum(lens[:i]), n) for i, n in enumerate(lens)]


def _exact_conv(case, st):
    x = st["x"].reshape(-1, case["C"])
    w, bias, keep = st["weight"].double(), st["bias"], case["W"] - 1
    out, state = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), st["state"].double()
    for (t0, n), slot in zip(_sequences(case), st["slots"].tolist()):
        for c0 in range(0, case["C"], 1024):
            c = slice(c0, min(case["C"], c0 + 1024))
            line = torch.cat([st["state"][slot, :, c].double(), x[t0:t0 + n, c].double()])
            if n:
                y = (line.unfold(0, keep + 1, 1) * w[c]).sum(-1)
                y = y if bias is None else y + bias[c].double()
                out[t0:t0 + n, c] = y * torch.sigmoid(y)
            state[slot, :, c] = line[n:]
    return dict(out=out.view(st["x"].shape), state=state)


def _exact_scan(case, st):
    di, ns = case["Di"], case["N"]
    x, z, dt = (st[k].reshape(-1, di) for k in ("x", "z", "dt"))
    bt, ct = (st[k].reshape(-1, ns) for k in ("Bt", "Ct"))
    seqs = _sequences(case)
    if sum(n for _, n in seqs) * di > 16384 * 5120:
        return None
    A, bias = st["A"].double(), st["dt_bias"].double()
    out, state = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), st["state"].double()
    start = torch.tensor([s for s, _ in seqs], device="cuda")
    length = [n for _, n in seqs]
    slots = st["slots"].long()
    for t in range(max(length)):
        live = torch.tensor([i for i, n in enumerate(length) if n > t])
        live = live.cuda() if len(live) < len(length) else slice(None)
        at, sl = start[live] + t, slots[live]
        xt, delta = x[at].double(), dt[at].double() + bias
        delta = torch.logaddexp(delta, torch.zeros_like(delta))
        h = torch.exp(delta[..., None] * A) * state[sl] + (delta * xt)[..., None] * bt[at].double()[:, None]
        state[sl] = h
        y = (h @ ct[at].double()[..., None])[..., 0] + st["D"].double() * xt
        g = z[at].double()
        out[at] = y * g * torch.sigmoid(g)
    return dict(out=out.view(st["x"].shape), state=state)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "cache":
        return {n: _exact_round_trip(st["new_" + n], case["bits"], case["dt"]) for n in ("k", "v")}
    if op == "attn":
        return _exact_attn(case, st)
    return (_exact_conv if op.startswith("conv") else _exact_scan)(case, st)


# --- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op in ("cache", "attn"):
        row = 2 * case["Hkv"] * (case["D"] * case["bits"] // 8 + case["D"] // _BLOCK)  # a token in the pages
    if op == "cache":
        n = case["tokens"]
        return dict(bytes=n * (2 * row + 8 * case["Hkv"] * case["D"] + 8), flops=12 * n * case["Hkv"] * case["D"])
    if op == "attn":
        lens, t, hq = _lengths(case), case["T"], case["Hkv"] * case["group"]
        pairs = sum(max(0, n - t + 1 + i) for n in lens for i in range(t))
        return dict(bytes=sum(lens) * row + 4 * case["B"] * t * hq * (case["D"] + 1), flops=4 * case["D"] * hq * pairs)
    step = op.endswith("step")
    n = case["B"] if step else case["nseq"]
    tokens = case["B"] * case["T"] if step else case["tokens"]
    if op.startswith("conv"):
        c, w = case["C"], case["W"]
        return dict(bytes=4 * tokens * c + 4 * n * (w - 1) * c + 2 * c * w, flops=(2 * w + 4) * tokens * c)
    di, ns = case["Di"], case["N"]
    return dict(bytes=tokens * (di * (8 + 2 * case["dt32"]) + 4 * ns) + 8 * n * di * ns + 4 * di * (ns + 2),
                flops=tokens * di * (7 * ns + 20))
