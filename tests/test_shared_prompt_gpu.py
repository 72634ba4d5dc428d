"""Adapters, rotated append and shared attention together: one attention layer
against its formulas in 64 bits, and the example that serves requests with them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_projection_append_and_attention_of_a_batch():
    """Three projections with adapters, the rotated append and the shared
    attention of one step, against the same chain in 64 bits from the dense
    products' outputs on. What the chain rounds: rotated queries and keys and
    the values to bf16 (2^-8 each), weights and output (2^-8 each); a score of
    `size` |q||k| moves by two roundings of it, so a weight by a factor within
    1 +- 4 * 2^-8 size, and the output by that times sum(p |v|), twice for the
    denominator."""
    import deepseek_v4_flash_gb300 as ds4
    import synth
    B, H, heads, kv, dim, page, S = 5, 128, 4, 2, 64, 16, 150
    lens = [S + x for x in (1, 20, 7, 33, 2)]
    g = torch.Generator().manual_seed(2)
    width = -(-max(lens) // page)
    table = torch.full((B, width), -1, dtype=torch.int32)
    whole = S // page
    table[:, :whole] = torch.arange(whole, dtype=torch.int32)
    at = whole
    for b in range(B):
        for p in range(whole, -(-lens[b] // page)):
            table[b, p] = at
            at += 1
    pool = torch.randn(2, at, page, kv, dim, generator=g).bfloat16()
    for b in range(1, B):
        pool[:, table[b, whole], :S % page] = pool[:, table[0, whole], :S % page]
    pool = pool.cuda()
    x = torch.from_numpy(np.ascontiguousarray(synth.gen_dense_x(3, B, H))).cuda()
    slots = torch.tensor([0, -1, 1, 1, 0], dtype=torch.int32).cuda()
    freq = 10000.0 ** -(torch.arange(0, dim, 2, dtype=torch.float32) / dim)
    rows, exact = {}, {}
    for i, (name, n) in enumerate((("q", heads), ("k", kv), ("v", kv))):
        dense = ds4.Dense(n * dim, H, torch.from_numpy(synth.gen_q8_matrix(4 + i, n * dim, H, 0.1)).cuda(), max_tokens=B)
        ad = ds4.Adapters(n * dim, H, 2, 12, "bf16", max_tokens=B)
        y = dense.forward(x).double().cpu()
        for s, r in enumerate((12, 5)):
            a, b = (torch.randn(r, H, generator=g) * H ** -0.5).bfloat16(), (torch.randn(n * dim, r, generator=g) * 0.2).bfloat16()
            ad.set(s, a.cuda(), b.cuda(), 0.5 + s)
            mine = (slots == s).cpu()
            y[mine] += (0.5 + s) * (x.cpu()[mine].double() @ a.double().T @ b.double().T)
        rows[name] = dense.forward(x, adapters=ad, slots=slots).view(B, 1, n, dim)
        exact[name] = y.view(B, n, dim)
    attn = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, max_seqs=B, max_tokens=B, max_shared_tokens=B))
    attn.debug_share()
    cache, kv_len = ds4.KVCache(pool[0], pool[1], table.cuda()), torch.tensor(lens, dtype=torch.int32).cuda()
    q = attn.append(cache, rows["k"], rows["v"], kv_len, rope=ds4.Rope(freq.cuda()), q=rows["q"])
    out = attn.decode(cache, q, kv_len, shared_len=torch.tensor([S], dtype=torch.int32).cuda())
    assert attn.device_error() == 0

    def turned(y, b):
        ang = (lens[b] - 1) * freq.double()
        lo, hi = y[..., :dim // 2], y[..., dim // 2:]
        return torch.cat([lo * ang.cos() - hi * ang.sin(), hi * ang.cos() + lo * ang.sin()], -1)
    u = 2.0 ** -8
    pool = pool.double().cpu()
    for b in range(B):
        pages = table[b, :-(-lens[b] // page)].long()
        k, v = (pool[i][pages].flatten(0, 1)[:lens[b]].clone() for i in range(2))
        k[-1], v[-1] = turned(exact["k"][b], b), exact["v"][b]
        qb = turned(exact["q"][b], b)
        for h in range(heads):
            kk, vv = k[:, h // 2], v[:, h // 2]
            s = kk @ qb[h] * dim ** -0.5
            p = torch.softmax(s, 0)
            ref = p @ vv
            size = float((kk.abs() @ qb[h].abs()).max()) * dim ** -0.5
            tol = u * ref.abs() + (2 * u + 8 * u * size) * (p @ vv.abs())
            assert ((out[b, 0, h].double().cpu() - ref).abs() <= tol).all(), (b, h)


def _args():
    rng = np.random.default_rng(3)
    return rng.integers(0, 1000, size=203).tolist(), [rng.integers(0, 1000, size=n).tolist() for n in (5, 17, 1, 30, 8)]


def test_example():
    """Serving with shared positions and without. Logits are not compared: the
    two attentions differ by their roundings, and a routing decision may flip on
    one of those. The first step's first attention is the same in both up to
    them: weights and output are rounded to bf16 in each (2^-8 of at most the
    largest |v| each time)."""
    from examples.shared_prompt import Server, generate
    system, prompts = _args()
    runs = []
    for share in (True, False):
        server = Server(5)
        server.attn.debug_share(share)
        first = []
        decode = server.attn.decode

        def watched(cache, q, kv_len, **kw):
            out = decode(cache, q, kv_len, **kw)
            if not first:
                first.append((out.clone(), cache.v.abs().max().item()))
            return out
        server.attn.decode = watched
        tokens, logits = generate(server, system, prompts, 8, share)
        assert not any(server.device_errors())
        assert len(tokens) == 5 and all(len(t) == 8 and all(0 <= x < 1000 for x in t) for t in tokens)
        assert all(torch.isfinite(x).all() for x in logits)
        runs.append((first[0], logits))
    ((a, top), la), ((b, _), lb) = runs
    assert torch.equal(la[0], lb[0])  # the prompts' own call is the same
    assert (a.float() - b.float()).abs().max() <= 4 * 2.0 ** -8 * top


def test_adapters_matter_in_the_example():
    """A request without an adapter is not changed by what the others' slots hold."""
    from examples.shared_prompt import Server, generate
    system, prompts = _args()
    one, two = Server(5), Server(5)
    for L in two.layers:
        for n in "qkvo":
            for s in range(3):
                L[n][1].clear(s)
    _, a = generate(one, system, prompts, 0)
    _, b = generate(two, system, prompts, 0)
    plain = [s < 0 for s in one.slot_of]
    for i, p in enumerate(plain):
        assert torch.equal(a[0][i], b[0][i]) == p
