"""Many requests behind one system prompt, each with its own low-rank adapter: a
small decoder with random weights whose projections, rotated append and decode
attention are called as a serving loop calls them.

    python examples/shared_prompt.py [--requests 6] [--tokens 16]

The system prompt is run once, without adapters. Its whole pages stand in every
request's block table; the page in which it ends is copied, for requests go on
writing there. The requests' own prompts run as one ragged call, then every
step runs one token of each: the projections carry each token's adapter
(Dense.forward(adapters=, slots=)), the append rotates queries and keys by their
positions on the way into the cache (Attention.append(rope=, q=)), and the
attention reads the system prompt's positions once for all requests
(Attention.decode(shared_len=)).
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import deepseek_v4_flash_gb300 as ds4  # noqa: E402
import synth  # noqa: E402


class Server:
    """`layers` x (RMSNorm, attention, MoE) over a paged cache. Request b uses
    adapter b % (n_adapters + 1) - 1: the first has none."""

    def __init__(self, requests=6, layers=2, vocab=1000, heads=8, kv_heads=2, dim=64, n_adapters=3, rank=8,
                 max_tokens=512, page_size=16, pages_each=24, seed=11):
        spec = synth.MICRO
        H = spec.hidden
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page_size
        self.requests = requests
        g = torch.Generator().manual_seed(seed)

        def projection(n_out, n_in, k, sigma):
            """A shared matrix and its adapters."""
            w = torch.from_numpy(synth.gen_q8_matrix(seed + k, n_out, n_in, sigma)).cuda()
            ad = ds4.Adapters(n_out, n_in, n_adapters, rank, "bf16", max_tokens=max_tokens)
            for i in range(n_adapters):
                r = rank - i  # ranks may differ
                ad.set(i, (torch.randn(r, n_in, generator=g) * n_in ** -0.5).bfloat16().cuda(),
                       (torch.randn(n_out, r, generator=g) * sigma).bfloat16().cuda(), scale=0.5)
            return ds4.Dense(n_out, n_in, w, max_tokens=max_tokens), ad
        self.emb = torch.randn(vocab, H, generator=g).cuda()
        self.head = ds4.Dense(vocab, H, torch.from_numpy(synth.gen_q8_matrix(seed, vocab, H, 0.1)).cuda(), max_tokens=max_tokens)
        n_pages = pages_each * (requests + 1)
        self.free = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.full((requests, pages_each * 2), -1, dtype=torch.int32)
        self.attn = ds4.Attention(ds4.AttentionDesc(heads, kv_heads, dim, "bf16", max_seqs=requests, max_tokens=max_tokens,
                                                    max_shared_tokens=requests))
        freq = 10000.0 ** -(torch.arange(0, dim, 2, dtype=torch.float32) / dim)
        self.rope = ds4.Rope(freq.cuda())
        self.slot_of = [b % (n_adapters + 1) - 1 for b in range(requests)]
        self.layers = []
        for i in range(layers):
            w = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in synth.gen_layer(spec, seed, i).items()}
            desc = ds4.LayerDesc(H, spec.n_experts, spec.top_k, spec.ffn, spec.n_shared, ds4.ROUTE_LEARNED, spec.vocab,
                                 ds4.FMT[spec.router_fmt], ds4.FMT[spec.routed_fmt], ds4.FMT[spec.shared_fmt],
                                 spec.route_scale, max_tokens)
            pool = torch.zeros(2, n_pages, page_size, kv_heads, dim, dtype=torch.bfloat16, device="cuda")
            self.layers.append(dict(
                moe=ds4.Layer(desc, w), q=projection(heads * dim, H, 10 * i + 2, 0.1),
                k=projection(kv_heads * dim, H, 10 * i + 3, 0.1), v=projection(kv_heads * dim, H, 10 * i + 4, 0.05),
                o=projection(H, heads * dim, 10 * i + 5, 0.05), pool=pool))
        self.shared = 0  # positions of the system prompt
        self.lens = [0] * requests

    def _grow(self, b, length):
        for p in range(-(-length // self.page)):
            if self.table[b, p] < 0:
                self.table[b, p] = self.free.pop()

    def _caches(self):
        table = self.table.cuda()
        return [ds4.KVCache(L["pool"][0], L["pool"][1], table) for L in self.layers]

    def _rows(self, tokens, slots, attend):
        """The decoder over rows of tokens; attend(layer, q, k, v) -> rows of heads."""
        h = self.emb[tokens.long()]
        n = torch.empty_like(h)
        for i, L in enumerate(self.layers):
            def proj(name, x):
                dense, adapters = L[name]
                return dense.forward(x, adapters=adapters, slots=slots)
            ds4.rmsnorm(h, n)
            q = proj("q", n).view(-1, self.heads, self.dim)
            k = proj("k", n).view(-1, self.kv_heads, self.dim)
            v = proj("v", n).view(-1, self.kv_heads, self.dim)
            o = attend(i, q, k, v)
            h += proj("o", o.float().reshape(-1, self.heads * self.dim))
            L["moe"].forward_rmsnorm(h, h)
        ds4.rmsnorm(h, n)
        return self.head.forward(n)

    def _ragged(self, runs, lens, slots):
        """Logits of all rows of ragged runs (lists of tokens), cached up to lens."""
        cu = torch.tensor(np.cumsum([0] + [len(r) for r in runs]), dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        tokens = torch.tensor([t for r in runs for t in r], dtype=torch.int32, device="cuda")
        rows = torch.tensor([s for r, s in zip(runs, slots) for _ in r], dtype=torch.int32, device="cuda")
        caches = self._caches()

        def attend(i, q, k, v):
            q = self.attn.append(caches[i], k, v, kv_len, cu_q=cu, rope=self.rope, q=q)
            return self.attn.prefill(caches[i], q, cu, kv_len)
        return self._rows(tokens, rows, attend), cu

    def system(self, tokens):
        """Run the system prompt once, and put it before every request."""
        self.shared = len(tokens)
        self._grow(0, self.shared)
        self._ragged([tokens], [self.shared], [-1])
        whole, rest = divmod(self.shared, self.page)
        for b in range(1, self.requests):
            self.table[b, :whole] = self.table[0, :whole]
            self._grow(b, self.shared)
            if rest:
                for L in self.layers:
                    L["pool"][:, int(self.table[b, whole]), :rest] = L["pool"][:, int(self.table[0, whole]), :rest]
        self.lens = [self.shared] * self.requests

    def prompts(self, prompts):
        """The requests' own prompts; logits [requests, vocab] after each."""
        self.lens = [n + len(p) for n, p in zip(self.lens, prompts)]
        for b, n in enumerate(self.lens):
            self._grow(b, n)
        logits, cu = self._ragged(prompts, self.lens, self.slot_of)
        return logits[cu[1:].long() - 1]

    def step(self, tokens, share=True):
        """One more token of every request; logits [requests, vocab]."""
        self.lens = [n + 1 for n in self.lens]
        for b, n in enumerate(self.lens):
            self._grow(b, n)
        kv_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        slots = torch.tensor(self.slot_of, dtype=torch.int32, device="cuda")
        shared = torch.tensor([self.shared], dtype=torch.int32, device="cuda") if share else None
        caches = self._caches()

        def attend(i, q, k, v):
            q = self.attn.append(caches[i], k, v, kv_len, rope=self.rope, q=q)
            return self.attn.decode(caches[i], q[:, None], kv_len, shared_len=shared)
        return self._rows(tokens, slots, attend)

    def device_errors(self):
        ops = [self.attn] + [L[n][k] for L in self.layers for n in "qkvo" for k in (0, 1)] + [L["moe"] for L in self.layers]
        return [x.device_error() for x in ops]


def generate(server, system, prompts, tokens, share=True):
    """Greedy tokens of every request, and the logits of each step."""
    server.system(system)
    logits = server.prompts(prompts)
    out, seen = [], [logits]
    for _ in range(tokens):
        nxt = logits.argmax(-1).int()
        out.append(nxt)
        logits = server.step(nxt, share)
        seen.append(logits)
    return (torch.stack(out, 1).tolist() if out else [[] for _ in prompts]), seen


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    rng = np.random.default_rng(3)
    server = Server(a.requests)
    system = rng.integers(0, 1000, size=203).tolist()
    prompts = [rng.integers(0, 1000, size=n).tolist() for n in rng.integers(1, 30, size=a.requests)]
    tokens, _ = generate(server, system, prompts, a.tokens)
    for b, t in enumerate(tokens):
        print("request", b, "adapter", server.slot_of[b], "->", t)
    print("device errors", sum(server.device_errors()))


if __name__ == "__main__":
    main()
