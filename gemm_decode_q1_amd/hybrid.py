"""A small hybrid decoder on the library's calls, as an example of their use:

    python -m gemm_decode_q1_amd.hybrid [--batch 8] [--prompt 300] [--tokens 64]
        [--pattern dda] [--conv 0] [--kv-bits 16]

Random Q1 weights.  Layers of the gated delta rule, of a selective state space
scan and of attention (over a prompt shared by the batch and each sequence's own
paged keys), each followed by the fused FFN; embedding and tied head from one
table.  A short causal convolution may stand before the scan and the delta rule,
and the keys and values may be held in 4 or 8 bits.  The prompt is run once: its
states are copied to every sequence, its keys and values are the shared prefix (in
4 or 8 bits: pages that stand in every sequence's table, but for the last one, which
answers go on in).  One decode step is a fixed sequence of launches, so it is
captured in a HIP graph and replayed.  There is no position encoding: between the
library's calls are only norms and activations.
"""
from __future__ import annotations

import argparse
import math
import time

import torch

from .decode import q1_delta_prefill, q1_delta_step, q1_prefix_attn, q1_sample
from .memory import PackedKV, q1_conv_prefill, q1_conv_step, q1_kv_attn, q1_kv_write, q1_scan_prefill, q1_scan_step
from .q1 import PackedQ1, q1_embed_rows, q1_ffn, q1_qmm


def random_q1(N: int, K: int, gen: torch.Generator) -> PackedQ1:
    """Random signs, scales for products of the size of the input."""
    packed = torch.randint(-2 ** 31, 2 ** 31, (N, K // 32), device="cuda", generator=gen, dtype=torch.int64).to(torch.int32)
    scales = (torch.rand(N, K // 128, device="cuda", generator=gen) + 0.5) * 2 / math.sqrt(K)
    return PackedQ1(packed, scales.half(), None, N, K)


def norm(x: torch.Tensor) -> torch.Tensor:
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class HybridDecoder:
    """``pattern``: one letter a layer, d (delta rule), s (state space scan) or a (attention).
    ``conv``: taps of the convolution before layers of kind d and s, 2 to 4, or 0 for none;
    ``kv_bits``: 16, or 8 or 4 for quantised pages; a scan has ``channels`` channels of ``N``
    numbers."""

    def __init__(self, pattern="dda", hidden=1024, inter=2048, vocab=8192, Hk=4, Hv=8, dim=128, Hq=8, Hkv=2, page=16,
                 seed=0, conv=0, kv_bits=16, channels=2048, N=16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pattern, self.hidden, self.vocab, self.page = pattern, hidden, vocab, page
        self.Hk, self.Hv, self.dim, self.Hq, self.Hkv = Hk, Hv, dim, Hq, Hkv
        self.conv, self.kv_bits, self.channels, self.N = conv, kv_bits, channels, N
        self.columns = {"d": (2 * Hk + Hv) * dim, "s": channels + 2 * N, "a": 0}  # first columns: those a convolution mixes
        rows = {"d": self.columns["d"] + 2 * Hv, "s": self.columns["s"] + 2 * channels, "a": (Hq + 2 * Hkv) * dim}
        wide = {"d": Hv * dim, "s": channels, "a": Hq * dim}
        self.layers = [dict(kind=c, proj=random_q1(rows[c], hidden, gen), out=random_q1(hidden, wide[c], gen),
                            gate=random_q1(inter, hidden, gen), up=random_q1(inter, hidden, gen),
                            down=random_q1(hidden, inter, gen)) for c in pattern]
        self.table = random_q1(vocab, hidden, gen)
        self.rate = torch.exp(torch.linspace(math.log(1e-3), math.log(1.0), Hv, device="cuda"))
        for layer in self.layers:
            columns = self.columns[layer["kind"]]
            if conv and columns:
                layer["taps"] = ((torch.rand(columns, conv, device="cuda", generator=gen) - 0.5) * 2 / math.sqrt(conv)).bfloat16()
        self.decay = -torch.arange(1, N + 1, dtype=torch.float32, device="cuda").repeat(channels, 1)  # the scan's A
        self.skip = torch.ones(channels, device="cuda")                                             # its D
        self.dt_bias = torch.linspace(-6.0, -2.0, channels, device="cuda")

    def _mix(self, y, layer, run):
        """The columns that come before the gates, through the convolution where there is one."""
        x = y[..., :self.columns[layer["kind"]]]
        return run(x, layer["taps"]) if "taps" in layer else x

    def _scan_inputs(self, x, y):
        """x, dt, A, B, C and what else a scan takes, as slices of the projection's rows."""
        c, n, at = self.channels, self.N, self.columns["s"]
        return ((x[..., :c], y[..., at:at + c], self.decay, x[..., c:c + n], x[..., c + n:]),
                dict(D=self.skip, z=y[..., at + c:], dt_bias=self.dt_bias))

    def _delta_inputs(self, x, y, lead):
        """q, k, v as slices of the (mixed) columns; log decay and write strength."""
        Hk, Hv, d = self.Hk, self.Hv, self.dim
        q, k, v = (x[..., a:a + n * d].view(*lead, n, d) for a, n in ((0, Hk), (Hk * d, Hk), (2 * Hk * d, Hv)))
        a, b = y[..., (2 * Hk + Hv) * d:].float().chunk(2, -1)
        return q, k, v, (-self.rate * torch.nn.functional.softplus(a)).view(*lead, Hv), torch.sigmoid(b).view(*lead, Hv)

    def _attn_inputs(self, y):
        y = y.view(y.shape[0], self.Hq + 2 * self.Hkv, self.dim)
        return y[:, :self.Hq], y[:, self.Hq:self.Hq + self.Hkv], y[:, self.Hq + self.Hkv:]

    def _finish(self, x, mixed, layer):
        """The layer's output projection and FFN, on the residual stream ``x`` (fp32)."""
        x = x + q1_qmm(mixed, layer["out"], torch.float32)
        return x + q1_ffn(norm(x), layer["gate"], layer["up"], layer["down"]).float()

    def prompt(self, ids: torch.Tensor) -> torch.Tensor:
        """Runs a prompt ``[P]``; returns its last token's logits and keeps its states, keys and values."""
        P, page = ids.numel(), self.page
        x = q1_embed_rows(ids, self.table, torch.float32)
        self.prompt_state, self.prompt_rows, self.prefix, self.prompt_tokens = {}, {}, {}, P
        cu = torch.tensor([0, P], dtype=torch.int32, device="cuda")
        for i, layer in enumerate(self.layers):
            y = q1_qmm(norm(x), layer["proj"])
            if "taps" in layer:
                self.prompt_rows[i] = torch.zeros(1, self.conv - 1, self.columns[layer["kind"]], dtype=y.dtype, device="cuda")
            x_in = self._mix(y, layer, lambda c, taps: q1_conv_prefill(c, taps, self.prompt_rows[i], cu))
            if layer["kind"] == "d":
                state = torch.zeros(1, self.Hv, self.dim, self.dim, device="cuda")
                mixed = q1_delta_prefill(*self._delta_inputs(x_in, y, (P,)), state, cu, l2norm=True)
                self.prompt_state[i] = state
            elif layer["kind"] == "s":
                state = torch.zeros(1, self.channels, self.N, device="cuda")
                given, more = self._scan_inputs(x_in, y)
                mixed = q1_scan_prefill(*given, state, cu, **more)
                self.prompt_state[i] = state
            elif self.kv_bits < 16:
                q, k, v = self._attn_inputs(y)
                n = -(-P // page)
                cache = PackedKV.empty(n, page, self.Hkv, self.dim, self.kv_bits)
                q1_kv_write(cache, k, v, torch.arange(P, dtype=torch.int32, device="cuda"))
                table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
                mixed = q1_kv_attn(q[None], cache, table, cu[1:])[0][0]
                self.prefix[i] = cache
            else:
                q, k, v = self._attn_inputs(y)
                # causal attention as P sequences over the same pages, of lengths 1..P
                n = -(-P // page)
                kv = torch.zeros(2, n * page, self.Hkv, self.dim, dtype=y.dtype, device="cuda")
                kv[0, :P], kv[1, :P] = k, v
                pages = kv.view(2, n, page, self.Hkv, self.dim)
                table = torch.arange(n, dtype=torch.int32, device="cuda").repeat(P, 1)
                lens = torch.arange(1, P + 1, dtype=torch.int32, device="cuda")
                mixed = q1_prefix_attn(q, None, None, pages[0], pages[1], table, lens)[0]
                self.prefix[i] = kv[:, :P]
            x = self._finish(x, mixed.flatten(1), layer)
        return q1_qmm(norm(x[-1:]), self.table, torch.float32)

    def begin(self, batch: int, most: int):
        """Room for ``batch`` answers of up to ``most`` tokens to the prompt."""
        per, page = -(-most // self.page), self.page
        self.state = {i: s.repeat(batch, *[1] * (s.dim() - 1)) for i, s in self.prompt_state.items()}
        self.rows = {i: r.repeat(batch, 1, 1) for i, r in self.prompt_rows.items()}
        self.most = most
        if self.kv_bits < 16:
            self._begin_quantised(batch, most)
            return
        self.pages = {i: torch.zeros(2, batch * per, page, self.Hkv, self.dim, dtype=kv.dtype, device="cuda")
                      for i, kv in self.prefix.items()}
        self.page_table = torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def _begin_quantised(self, batch: int, most: int):
        """The prompt's full pages stand in every table; each sequence has its own copy of a
        last one that is not full, and pages for its answer."""
        page, full = self.page, self.prompt_tokens // self.page
        part = self.prompt_tokens - full * page
        per = -(-(part + most) // page)
        own = full + torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
        self.page_table = torch.cat([torch.arange(full, dtype=torch.int32, device="cuda").expand(batch, -1), own], 1).contiguous()
        self.lens = torch.full((batch,), self.prompt_tokens, dtype=torch.int32, device="cuda")
        self.pages = {}
        for i, old in self.prefix.items():
            new = PackedKV.empty(full + batch * per, page, self.Hkv, self.dim, self.kv_bits)
            for to, of in zip((new.k, new.v, new.k_scales, new.v_scales), (old.k, old.v, old.k_scales, old.v_scales)):
                to[:full] = of[:full]
                if part:
                    to[own[:, 0].long()] = of[full]
            self.pages[i] = new

    def logits(self, ids: torch.Tensor) -> torch.Tensor:
        """One decode step of the batch: takes a token of each sequence (at most
        ``most`` times in all), returns the logits after it."""
        x = q1_embed_rows(ids, self.table, torch.float32)
        B = ids.numel()
        at = self.lens.long()
        slot = self.page_table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page
        self.lens += 1
        for i, layer in enumerate(self.layers):
            y = q1_qmm(norm(x), layer["proj"])
            x_in = self._mix(y, layer, lambda c, taps: q1_conv_step(c[:, None], taps, self.rows[i])[:, 0])
            if layer["kind"] == "d":
                mixed = q1_delta_step(*self._delta_inputs(x_in, y, (B, 1)), self.state[i], l2norm=True)
            elif layer["kind"] == "s":
                given, more = self._scan_inputs(x_in[:, None], y[:, None])
                mixed = q1_scan_step(*given, self.state[i], **more)
            elif self.kv_bits < 16:
                q, k, v = self._attn_inputs(y)
                q1_kv_write(self.pages[i], k, v, slot.int())
                mixed = q1_kv_attn(q[:, None], self.pages[i], self.page_table, self.lens)[0]
            else:
                q, k, v = self._attn_inputs(y)
                pages, prefix = self.pages[i], self.prefix[i]
                pages.view(2, -1, self.Hkv, self.dim)[0].index_copy_(0, slot, k)
                pages.view(2, -1, self.Hkv, self.dim)[1].index_copy_(0, slot, v)
                mixed = q1_prefix_attn(q, prefix[0], prefix[1], pages[0], pages[1], self.page_table, self.lens)[0]
            x = self._finish(x, mixed.reshape(B, -1), layer)
        return q1_qmm(norm(x), self.table, torch.float32)

    def generate(self, ids: torch.Tensor, batch: int, tokens: int, seed=0, graph=True, **filters):
        """``batch`` sampled answers ``[batch, tokens]`` to the prompt ``ids``, and
        their log-probabilities; ``filters`` as for ``q1_sample``."""
        first = self.prompt(ids).expand(batch, -1).contiguous()
        self.begin(batch, max(tokens, 2))
        u = torch.rand(tokens, batch, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
        token, logprob = q1_sample(first, u[0], **filters)
        got = [(token.clone(), logprob.clone())]
        draw = torch.empty(batch, device="cuda")

        def step():
            q1_sample(self.logits(token), draw, tokens=token, logprob=logprob, **filters)

        replay = step
        for t in range(1, tokens):
            draw.copy_(u[t])
            if graph and t == 2:  # (the first step has run eagerly, so every workspace is there)
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    step()
                replay = captured.replay
            replay()
            got.append((token.clone(), logprob.clone()))
        return torch.stack([g[0] for g in got], 1), torch.stack([g[1] for g in got], 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--pattern", default="dda", help="a letter a layer: d delta rule, s state space scan, a attention")
    ap.add_argument("--conv", type=int, default=0, help="taps of the short convolution, 2 to 4")
    ap.add_argument("--kv-bits", type=int, default=16, choices=(4, 8, 16))
    a = ap.parse_args()
    model = HybridDecoder(pattern=a.pattern, conv=a.conv, kv_bits=a.kv_bits)
    ids = torch.randint(0, model.vocab, (a.prompt,), device="cuda", dtype=torch.int32)
    filters = dict(temperature=torch.full((a.batch,), 0.8, device="cuda"), top_p=torch.full((a.batch,), 0.9, device="cuda"),
                   top_k=torch.full((a.batch,), 50, dtype=torch.int32, device="cuda"))
    for _ in range(2):  # the first pass sets everything up
        torch.cuda.synchronize()
        began = time.perf_counter()
        tokens, logprobs = model.generate(ids, a.batch, a.tokens, **filters)
        torch.cuda.synchronize()
        took = time.perf_counter() - began
    print("first tokens:", tokens[:, :8].tolist())
    print(f"{a.batch} answers of {a.tokens} tokens to a prompt of {a.prompt}: {1e3 * took:.1f} ms, "
          f"mean logprob {logprobs.mean().item():.2f}")


if __name__ == "__main__":
    main()
