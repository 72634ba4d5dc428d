"""Speculative decoding of a small decoder with random weights: the attention
operators, the dense products, the MoE layers and the sampling steps together,
as a serving loop calls them.

    python examples/speculative_decode.py [--tokens 64] [--temperature 0.8]

A step of every sequence: the drafter (a look-up of what followed the same two
tokens earlier in the sequence, sure of its guesses) proposes up to `drafts`
tokens; the decoder runs the last accepted token and the drafts as new tokens
of one call (append to the paged cache, attention over it, MoE), the output
head's logits become probabilities, and ds4moe_verify_drafts keeps the drafts
that the decoder would have drawn and draws the next token. The cache needs no
undoing: rejected rows lie past the sequence's length and the next step
overwrites them.
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


class Decoder:
    """`layers` x (RMSNorm, attention, MoE) over a paged cache; no position
    code, weights random. The rows of a call are [n_seq, n_new] tokens (decode)
    or ragged prompts (prefill)."""

    def __init__(self, layers=2, vocab=1000, heads=8, kv_heads=1, dim=64, window=0, n_sink=0, seqs=4, max_tokens=512,
                 pages=64, page_size=16, seed=7):
        spec = synth.MICRO
        H = spec.hidden
        self.H, self.heads, self.kv_heads, self.dim, self.vocab = H, heads, kv_heads, dim, vocab

        def dense(n_out, n_in, k, sigma):
            w = torch.from_numpy(synth.gen_q8_matrix(seed + k, n_out, n_in, sigma)).cuda()
            return ds4.Dense(n_out, n_in, w, max_tokens=max_tokens)
        g = torch.Generator().manual_seed(seed)
        self.emb = torch.randn(vocab, H, generator=g).cuda()
        self.head = dense(vocab, H, 1, 0.1)
        self.layers = []
        per_seq = pages // seqs
        table = torch.arange(pages, dtype=torch.int32)[torch.randperm(pages, generator=g)]
        self.table = table[:per_seq * seqs].view(seqs, per_seq).contiguous().cuda()
        # one handle for all layers: they run one after another
        self.attn = ds4.Attention(ds4.AttentionDesc(heads, kv_heads, dim, "bf16", window, n_sink, None, seqs, max_tokens))
        for i in range(layers):
            w = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in synth.gen_layer(spec, seed, i).items()}
            desc = ds4.LayerDesc(H, spec.n_experts, spec.top_k, spec.ffn, spec.n_shared, ds4.ROUTE_LEARNED, spec.vocab,
                                 ds4.FMT[spec.router_fmt], ds4.FMT[spec.routed_fmt], ds4.FMT[spec.shared_fmt],
                                 spec.route_scale, max_tokens)
            pool = torch.zeros(2, pages, page_size, kv_heads, dim, dtype=torch.bfloat16, device="cuda")
            self.layers.append(dict(
                moe=ds4.Layer(desc, w), q=dense(heads * dim, H, 10 * i + 2, 0.1), k=dense(kv_heads * dim, H, 10 * i + 3, 0.1),
                v=dense(kv_heads * dim, H, 10 * i + 4, 0.05), o=dense(H, heads * dim, 10 * i + 5, 0.05),
                cache=ds4.KVCache(pool[0], pool[1], self.table)))

    def _rows(self, tokens, kv_len, shape, cu_q):
        h = self.emb[tokens.reshape(-1).long()]
        n = torch.empty_like(h)
        for L in self.layers:
            ds4.rmsnorm(h, n)
            q = L["q"].forward(n).bfloat16().view(*shape, self.heads, self.dim)
            k = L["k"].forward(n).view(*shape, self.kv_heads, self.dim)
            v = L["v"].forward(n).view(*shape, self.kv_heads, self.dim)
            self.attn.append(L["cache"], k, v, kv_len, cu_q=cu_q)
            if cu_q is None:
                o = self.attn.decode(L["cache"], q, kv_len)
            else:
                o = self.attn.prefill(L["cache"], q, cu_q, kv_len)
            h += L["o"].forward(o.float().view(-1, self.heads * self.dim))
            L["moe"].forward_rmsnorm(h, h)
        ds4.rmsnorm(h, n)
        return self.head.forward(n)

    def prefill(self, prompts):
        """Logits [n_seq, vocab] after each prompt (lists of token ids)."""
        cu = np.cumsum([0] + [len(p) for p in prompts])
        cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kv_len = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device="cuda")
        logits = self._rows(tokens, kv_len, (len(tokens),), cu_q)
        return logits[torch.from_numpy(cu[1:] - 1).cuda()]

    def decode(self, tokens, kv_len):
        """Logits [n_seq, n_new, vocab] of new tokens; kv_len counts them."""
        logits = self._rows(tokens, kv_len, tuple(tokens.shape), None)
        return logits.view(*tokens.shape, self.vocab)

    def device_errors(self):
        return [L["moe"].device_error() for L in self.layers] + [self.attn.device_error()]


def look_up(seq, drafts):
    """What followed the last earlier occurrence of the sequence's two last tokens."""
    for i in range(len(seq) - 3, -1, -1):
        if seq[i:i + 2] == seq[-2:]:
            return seq[i + 2:i + 2 + drafts]
    return []


def generate(model, prompts, tokens, drafts=3, temperature=0.8, seed=1):
    """Extends every prompt by at least `tokens` tokens; returns the sequences
    and (drafted, accepted) totals."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(prompts)
    seqs = [list(p) for p in prompts]
    probs = ds4.token_probs(model.prefill(prompts), temperature)
    none = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    _, first = ds4.verify_drafts(probs[:, None].contiguous(), None, none, none.float(),
                                 torch.rand(B, generator=g, device="cuda"))
    for s, t in zip(seqs, first[:, 0].tolist()):
        s.append(t)
    drafted = accepted = 0
    goal = [len(p) + tokens for p in prompts]
    while any(len(s) < n for s, n in zip(seqs, goal)):
        guess = [look_up(s, drafts) for s in seqs]
        count = torch.tensor([len(x) for x in guess], dtype=torch.int32, device="cuda")
        draft = torch.tensor([x + [0] * (drafts - len(x)) for x in guess], dtype=torch.int32, device="cuda")
        last = torch.tensor([[s[-1]] for s in seqs], dtype=torch.int32, device="cuda")
        # the last token is not in the cache yet: it and the drafts are the new tokens
        kv_len = torch.tensor([len(s) + drafts for s in seqs], dtype=torch.int32, device="cuda")
        logits = model.decode(torch.cat([last, draft], 1), kv_len)
        probs = ds4.token_probs(logits, temperature, out=logits)
        n, out = ds4.verify_drafts(probs, None, draft, torch.rand(B, drafts, generator=g, device="cuda"),
                                   torch.rand(B, generator=g, device="cuda"), n_draft=count)
        for s, k, row in zip(seqs, n.tolist(), out.tolist()):
            s.extend(row[:k + 1])
        drafted += int(count.sum())
        accepted += int(n.sum())
    return seqs, drafted, accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    model = Decoder()
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, 1000, size=n).tolist() for n in (5, 17, 40, 1)]
    seqs, drafted, accepted = generate(model, prompts, a.tokens, temperature=a.temperature)
    for p, s in zip(prompts, seqs):
        print(len(p), "->", len(s), "tokens:", s[len(p):len(p) + 12], "...")
    print("drafted", drafted, "accepted", accepted, "device errors", model.device_errors())


if __name__ == "__main__":
    main()
