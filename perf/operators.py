"""The operators between the Q1 projections of a decode step, as measured cases.

Four calls: the gated delta rule for single tokens (``q1_delta_step``) and for
whole prompts (``q1_delta_prefill``), attention of a decode batch over a shared
prefix (``q1_prefix_attn``) and the sampler of the tied head's logits
(``q1_sample``).  ``run`` computes them in plain torch operations in 32 bits,
or, where ``own`` is true, through this repository's package.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_EPS = 1e-6       # added to the squared norm of q and k
_CHUNK = 64       # tokens the plain prompt form takes at a time
_UNIT = 2.0 ** 40  # sampling weights are whole multiples of 2^-40


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # one user's next token: 48 heads' states, where latency counts
        dict(name="step one sequence", op="step", B=1, T=1, Hk=16, Hv=48, Dk=128, Dv=128, dt="bf16", l2=True),
        # a full batch of packed activation rows (8)
        dict(name="step eight sequences", op="step", B=8, T=1, Hk=16, Hv=48, Dk=128, Dv=128, dt="bf16", l2=True),
        # a large batch that checks three drafted tokens a sequence, keys normalised beforehand
        dict(name="step drafted tokens", op="step", B=61, T=3, Hk=16, Hv=48, Dk=128, Dv=128, dt="f16", l2=False),
        # a short odd prompt
        dict(name="prefill short", op="prefill", tokens=77, nseq=1, Hk=16, Hv=48, Dk=128, Dv=128, dt="bf16", l2=True),
        # a ragged batch of prompts, single tokens among them
        dict(name="prefill ragged", op="prefill", tokens=4099, nseq=7, Hk=8, Hv=32, Dk=128, Dv=128, dt="f16", l2=True),
        # one long prompt
        dict(name="prefill long", op="prefill", tokens=16384, nseq=1, Hk=16, Hv=48, Dk=128, Dv=128, dt="bf16", l2=True),
        # a few users of one short system prompt
        dict(name="attn short prefix", op="attn", B=4, Hkv=4, group=6, D=128, P=519, most=40, page=16, dt="bf16"),
        # a batch of answers to one document, some of them not begun
        dict(name="attn batch", op="attn", B=32, Hkv=4, group=6, D=256, P=8201, most=700, page=64, dt="bf16"),
        # eight users of one very long context
        dict(name="attn long prefix", op="attn", B=8, Hkv=8, group=4, D=128, P=65537, most=2000, page=48, dt="f16"),
        # one row of the tied head's 152064 logits
        dict(name="sample one row", op="sample", B=1, V=152064, dt="f32", kind="mixed"),
        # a batch of packed rows
        dict(name="sample eight rows", op="sample", B=8, V=152064, dt="bf16", kind="mixed"),
        # a large batch, rows with every filter and with none
        dict(name="sample large batch", op="sample", B=192, V=152064, dt="f32", kind="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["step", "prefill", "attn", "sample"])
    if op == "sample":
        return dict(op=op, B=_log(rng, 1, 160), V=_log(rng, 100, 152064), dt=rng.choice(["f32", "bf16", "f16"]),
                    kind=rng.choice(["mixed", "plain", "greedy", "top-k", "top-p"]))
    if op == "attn":
        c = dict(op=op, B=_log(rng, 1, 48), Hkv=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 3, 4, 6, 8]),
                 D=rng.choice([64, 128, 256]), P=_log(rng, 1, 65536), most=_log(rng, 1, 2000),
                 page=rng.choice([1, 16, 17, 48, 64]), dt=rng.choice(["bf16", "f16"]))
        while c["B"] * c["Hkv"] * c["group"] * c["D"] * (c["P"] + c["most"]) > 8 * 8 * 4 * 128 * 67537:
            c["P"] = c["P"] // 2 + 1
            c["B"] = c["B"] // 2 + 1
        return c
    hk, hv = rng.choice([(16, 48), (8, 32), (4, 12), (2, 2), (3, 3), (1, 6)])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128)])
    c = dict(op=op, Hk=hk, Hv=hv, Dk=dk, Dv=dv, dt=rng.choice(["bf16", "f16"]), l2=rng.random() < 0.7)
    if op == "step":
        return dict(c, B=_log(rng, 1, 60), T=rng.choice([1, 1, 1, 2, 3, 4]))
    tokens = _log(rng, 1, 12000)
    return dict(c, tokens=tokens, nseq=_log(rng, 1, 16))


def _lengths(case):
    """Lengths of a ragged batch: from the case alone, so that its work is known."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "attn":
        got = [min(case["most"], int(case["most"] * r.random() ** 1.5) + (r.random() < 0.9)) for _ in range(case["B"])]
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


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + _EPS)


def _delta_inputs(case, g, lead):
    """q, k, v as column slices of one projection's rows; decays from 0.999 to
    a fast forgetting by head; write strengths in (0, 1)."""
    hk, hv, dk, dv, dt = case["Hk"], case["Hv"], case["Dk"], case["Dv"], _DT[case["dt"]]
    x = _randn(g, *lead, 2 * hk * dk + hv * dv)
    if not case["l2"]:
        qk = _unit(x[..., :2 * hk * dk].unflatten(-1, (2 * hk, dk))).flatten(-2)
        x = torch.cat([qk, x[..., 2 * hk * dk:]], -1)
    x = x.to(dt)
    q = x[..., :hk * dk].unflatten(-1, (hk, dk))
    k = x[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
    v = x[..., 2 * hk * dk:].unflatten(-1, (hv, dv))
    rate = torch.exp(torch.linspace(math.log(1e-3), math.log(1.5), hv, device="cuda"))
    decay = -rate * torch.nn.functional.softplus(_randn(g, *lead, hv) + 0.5)
    beta = torch.sigmoid(_randn(g, *lead, hv))
    return dict(q=q, k=k, v=v, g=decay, beta=beta)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("step", "prefill"):
        n = case["B"] if op == "step" else case["nseq"]
        lead = (case["B"], case["T"]) if op == "step" else (case["tokens"],)
        st = dict(_delta_inputs(case, g, lead), op=op, l2=case["l2"])
        pool = n + 3  # a pool of states, of which this batch holds some in any order
        st["state"] = 0.2 * _randn(g, pool, case["Hv"], case["Dk"], case["Dv"])
        st["slots"] = torch.randperm(pool, device="cuda", generator=g)[:n].to(torch.int32)
        if op == "prefill":
            st["lens"] = _lengths(case)
            st["cu"] = torch.tensor([0] + list(np.cumsum(st["lens"])), dtype=torch.int32).cuda()
        return st
    if op == "attn":
        b, hkv, grp, d, dt = case["B"], case["Hkv"], case["group"], case["D"], _DT[case["dt"]]
        lens = _lengths(case)
        per = -(-case["most"] // case["page"])
        st = dict(op=op, q=(1.5 * _randn(g, b, hkv * grp, d)).to(dt),
                  kp=_randn(g, case["P"], hkv, d).to(dt), vp=_randn(g, case["P"], hkv, d).to(dt),
                  kc=_randn(g, b * per + 2, case["page"], hkv, d).to(dt),
                  vc=_randn(g, b * per + 2, case["page"], hkv, d).to(dt))
        st["table"] = torch.randperm(b * per + 2, device="cuda", generator=g)[:b * per].to(torch.int32).view(b, per)
        st["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        return st
    b, v = case["B"], case["V"]
    # a language model's logits: a broad body, and some dozens of likely tokens
    logits = 2.0 * _randn(g, b, v)
    hot = torch.randint(0, v, (b, 48), device="cuda", generator=g)
    logits.scatter_(1, hot, 6.0 + 3.0 * _randn(g, b, 48))
    st = dict(op=op, logits=logits.to(_DT[case["dt"]]), u=_rand(g, b))
    kind = case["kind"]
    row = torch.arange(b, device="cuda")
    on = {"mixed": lambda m: row % 4 == m, "plain": lambda m: row < 0, "greedy": lambda m: row < 0,
          "top-k": lambda m: (row >= 0) & (m == 1), "top-p": lambda m: (row >= 0) & (m == 2)}[kind]
    both = (row % 4 == 0) if kind == "mixed" else row < 0  # rows with every filter at once
    st["temperature"] = torch.zeros(b, device="cuda") if kind == "greedy" else 0.5 + 0.8 * _rand(g, b)
    ks = torch.randint(1, 200, (b,), device="cuda", generator=g).to(torch.int32)
    st["top_k"] = torch.where(on(1) | both, ks, torch.zeros_like(ks))
    st["top_p"] = torch.where(on(2) | both, 0.7 + 0.29 * _rand(g, b), torch.ones(b, device="cuda"))
    st["min_p"] = torch.where(both, 0.1 * _rand(g, b), torch.zeros(b, device="cuda"))
    return st


# --- plain forms ------------------------------------------------------------

def _delta_operands(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    if st["l2"]:
        q, k = _unit(q), _unit(k)
    rep = v.shape[-2] // k.shape[-2]
    return q.repeat_interleave(rep, -2) * k.shape[-1] ** -0.5, k.repeat_interleave(rep, -2), v


def _plain_step(st):
    q, k, v = _delta_operands(st)
    slots = st["slots"].long()
    S = st["state"][slots]
    out = torch.empty_like(v)
    for t in range(q.shape[1]):
        S = S * st["g"][:, t].exp()[..., None, None]
        d = (v[:, t] - (S * k[:, t, :, :, None]).sum(-2)) * st["beta"][:, t, :, None]
        S = S + k[:, t, :, :, None] * d[:, :, None, :]
        out[:, t] = (S * q[:, t, :, :, None]).sum(-2)
    st["state"][slots] = S
    return dict(out=out.to(st["v"].dtype), state=st["state"])


def _plain_prefill(st):
    q, k, v = _delta_operands(st)
    lens = torch.tensor(st["lens"])
    n, C = len(st["lens"]), _CHUNK
    chunks = max(1, -(-max(st["lens"]) // C))
    pos = torch.arange(chunks * C)
    inside = (pos[None] < lens[:, None]).cuda()
    at = (st["cu"][:-1].long()[:, None] + pos.cuda()[None]).clamp(max=q.shape[0] - 1)

    def chunked(x):  # [tokens, heads, ...] -> [sequence, head, chunk, C, ...], zeros past the end
        x = torch.where(inside.view(n, -1, *[1] * (x.dim() - 1)), x[at], torch.zeros((), device="cuda"))
        return x.unflatten(1, (chunks, C)).movedim(3, 1)

    q, k, v, beta = chunked(q), chunked(k), chunked(v), chunked(st["beta"])
    G = chunked(st["g"]).cumsum(-1)
    low = torch.ones(C, C, device="cuda").tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]) * low) * low
    A = (k @ k.transpose(-1, -2)) * D * beta[..., None]
    A = A * low.tril(-1)
    T = torch.eye(C, device="cuda").expand(A.shape).clone()
    for i in range(1, C):  # row i of the inverse from the rows above it
        T[..., i:i + 1, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])
    P = (q @ k.transpose(-1, -2)) * D
    eG, left = G.exp()[..., None], torch.exp(G[..., -1:] - G)[..., None]
    slots = st["slots"].long()
    S = st["state"][slots]
    out = torch.empty_like(v)
    for c in range(chunks):
        d = T[:, :, c] @ ((v[:, :, c] - eG[:, :, c] * (k[:, :, c] @ S)) * beta[:, :, c, :, None])
        out[:, :, c] = eG[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ d
        S = eG[:, :, c, -1:] * S + (k[:, :, c] * left[:, :, c]).transpose(-1, -2) @ d
    st["state"][slots] = S
    rows = out.movedim(1, 3).flatten(1, 2)[inside]
    return dict(out=rows.to(st["v"].dtype), state=st["state"])


def _plain_attn(st):
    q, lens, table = st["q"].float(), st["lens"].long(), st["table"].long()
    b, hq, d = q.shape
    hkv = st["kp"].shape[1]
    q = q.view(b, hkv, hq // hkv, d) * d ** -0.5
    kp, vp = (st[x].float().movedim(0, 1) for x in ("kp", "vp"))                    # [Hkv, P, D]
    kc, vc = (st[x][table].flatten(1, 2).float().movedim(1, 2) for x in ("kc", "vc"))  # [B, Hkv, L, D]
    sp = (q.movedim(1, 0).flatten(1, 2) @ kp.transpose(-1, -2)).unflatten(1, (b, -1)).movedim(0, 1)
    sc = q @ kc.transpose(-1, -2)
    gone = torch.arange(kc.shape[2], device="cuda")[None] >= lens[:, None]
    sc = sc.masked_fill(gone[:, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1), sc.amax(-1))[..., None]
    sp, sc = torch.exp(sp - m), torch.exp(sc - m)
    total = sp.sum(-1) + sc.sum(-1)
    o = (sp.movedim(1, 0).flatten(1, 2) @ vp).unflatten(1, (b, -1)).movedim(0, 1) + sc @ vc
    out = (o / total[..., None]).reshape(b, hq, d)
    return dict(out=out.to(st["q"].dtype), lse=(m[..., 0] + total.log()).reshape(b, hq))


def _plain_sample(st):
    x = st["logits"].float()
    b, v = x.shape
    T = st["temperature"][:, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(T > 0, T, torch.ones_like(T)))
    s, order = torch.sort(x, dim=-1, descending=True, stable=True)
    es = e.gather(1, order)
    ws = (es * _UNIT).to(torch.int64)
    rank = torch.arange(v, device="cuda")[None]
    k = st["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (T <= 0), torch.where(T <= 0, 1, v), k)
    ws = torch.where(rank < k, ws, 0)
    before = ws.cumsum(-1)
    bound = (st["top_p"].double()[:, None] * before[:, -1:].double()).to(torch.int64).clamp(min=1)
    bound = torch.where(st["top_p"][:, None] < 1, bound, before[:, -1:] + 1)
    keep = (before - ws < bound) & (es >= st["min_p"][:, None])
    w = torch.zeros_like(ws).scatter_(1, order, torch.where(keep, ws, 0))
    upto = w.cumsum(-1)
    total = upto[:, -1]
    r = (st["u"].double() * total.double()).to(torch.int64)
    token = (upto <= r[:, None]).sum(-1)
    mine = w.gather(1, token[:, None])[:, 0]
    return dict(token=token, logprob=torch.log((mine.double() / total.double()).float()))


_PLAIN = dict(step=_plain_step, prefill=_plain_prefill, attn=_plain_attn, sample=_plain_sample)


def run(state):
    st = state
    if not own:
        return _PLAIN[st["op"]](st)
    import gemm_decode_q1_amd as Q
    if st["op"] == "step":
        out = Q.q1_delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["slots"],
                              l2norm=st["l2"])
        return dict(out=out, state=st["state"])
    if st["op"] == "prefill":
        out = Q.q1_delta_prefill(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["cu"], st["slots"],
                                 l2norm=st["l2"])
        return dict(out=out, state=st["state"])
    if st["op"] == "attn":
        out, lse = Q.q1_prefix_attn(st["q"], st["kp"], st["vp"], st["kc"], st["vc"], st["table"], st["lens"])
        return dict(out=out, lse=lse)
    token, logprob = Q.q1_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                 top_p=st["top_p"], min_p=st["min_p"])
    return dict(token=token, logprob=logprob)


# --- the same from the definitions, in 64 bits --------------------------------

def _exact_delta(case, st):
    step = case["op"] == "step"
    q, k, v, g, beta = (st[x].double() for x in ("q", "k", "v", "g", "beta"))
    if case["l2"]:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + _EPS)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + _EPS)
    head = torch.arange(case["Hv"], device="cuda") // (case["Hv"] // case["Hk"])
    if step:
        lens = [case["T"]] * case["B"]
        q, k, v, g, beta = (x.flatten(0, 1) for x in (q, k, v, g, beta))
    else:
        lens = _lengths(case)
    first = torch.tensor([0] + list(np.cumsum(lens)))[:-1].cuda()
    length = torch.tensor(lens).cuda()
    slots = st["slots"].long()
    S = st["state"].double()[slots].transpose(-1, -2).contiguous()  # [sequence, head, Dv, Dk]
    out = torch.zeros_like(v)
    for t in range(max(lens)):
        seq = (length > t).nonzero()[:, 0] if len(lens) > 1 else torch.zeros(1, dtype=torch.long, device="cuda")
        tok = first[seq] + t
        whole = len(lens) == 1 or step  # every sequence has a token t
        s = S if whole else S[seq]
        kt, qt = k[tok][:, head], q[tok][:, head]
        s = s * torch.exp(g[tok])[..., None, None]
        err = v[tok] - (s @ kt[..., None])[..., 0]
        s = s + (beta[tok][..., None] * err)[..., None] * kt[..., None, :]
        out[tok] = (s @ qt[..., None])[..., 0] / math.sqrt(case["Dk"])
        if whole:
            S = s
        else:
            S[seq] = s
    state = st["state"].double()
    state[slots] = S.transpose(-1, -2)
    return dict(out=out.view(st["v"].shape), state=state)


def _exact_attn(case, st):
    b, hq, d = st["q"].shape
    outs, lses = [], []
    for i, n in enumerate(_lengths(case)):
        pages = st["table"][i].long()
        k = torch.cat([st["kp"], st["kc"][pages].flatten(0, 1)[:n]]).double()
        v = torch.cat([st["vp"], st["vc"][pages].flatten(0, 1)[:n]]).double()
        q = st["q"][i].double().view(case["Hkv"], case["group"], d)
        s = q @ k.permute(1, 2, 0).contiguous() / math.sqrt(d)
        lse = torch.logsumexp(s, -1)
        outs.append((torch.exp(s - lse[..., None]) @ v.transpose(0, 1).contiguous()).reshape(hq, d))
        lses.append(lse.reshape(hq))
    return dict(out=torch.stack(outs), lse=torch.stack(lses))


def _exact_sample(case, st):
    """Row by row; the drawn token has no value in 64 bits (it is a choice), its
    log probability has one."""
    got = []
    x = st["logits"].double().cpu().numpy()
    par = {n: st[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    for i in range(case["B"]):
        row, T = x[i], par["temperature"][i]
        if T <= 0:
            got.append(0.0)
            continue
        e = np.exp((row - row.max()) / T)
        w = np.floor(e * _UNIT)
        live = np.flatnonzero(w > 0)
        order = live[np.lexsort((live, -row[live]))]
        if par["top_k"][i] > 0:
            order = order[:int(par["top_k"][i])]
        c = np.cumsum(w[order])
        if par["top_p"][i] < 1:
            order = order[(c - w[order]) < max(1.0, np.floor(par["top_p"][i] * c[-1]))]
        order = np.sort(order[e[order] >= par["min_p"][i]])
        c = np.cumsum(w[order])
        j = int(np.searchsorted(c, np.floor(par["u"][i] * c[-1]), side="right"))
        got.append(math.log(w[order[j]] / c[-1]))
    return dict(token=None, logprob=torch.tensor(got, dtype=torch.float64))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("step", "prefill"):
        return _exact_delta(case, st)
    return (_exact_attn if case["op"] == "attn" else _exact_sample)(case, st)


# --- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "sample":
        size = 4 if case["dt"] == "f32" else 2
        return dict(bytes=case["B"] * (case["V"] * size + 32), flops=4 * case["B"] * case["V"])
    if op == "attn":
        tail, hq = sum(_lengths(case)), case["Hkv"] * case["group"]
        return dict(bytes=4 * (case["P"] + tail) * case["Hkv"] * case["D"] + 4 * case["B"] * hq * (case["D"] + 1),
                    flops=4 * case["D"] * hq * (case["B"] * case["P"] + tail))
    n = case["B"] if op == "step" else case["nseq"]
    tokens = case["B"] * case["T"] if op == "step" else case["tokens"]
    state = case["Hv"] * case["Dk"] * case["Dv"]
    row = 2 * (2 * case["Hk"] * case["Dk"] + 2 * case["Hv"] * case["Dv"]) + 8 * case["Hv"]
    return dict(bytes=8 * n * state + tokens * row, flops=7 * tokens * state)
