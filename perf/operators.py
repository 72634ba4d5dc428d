"""The operators of one decoding step around the MoE layer, as cases to measure.

A paged key-value cache is written (``append``), read by new tokens
(``decode``: one or a few drafted tokens per sequence; ``prefill``: ragged
runs of many tokens, with a sliding window and first tokens that stay
visible), the output head's logits become probabilities (``probs``), and
drafted tokens are checked against them (``verify``).

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, 64 where a border decides an integer), or, with ``own`` set, through
the package's public entry points. ``exact`` evaluates the definition in 64
bits, written apart from the plain form.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one user's chat turn early on: a single sequence, short cache, latency counts
        dict(name="decode-single", op="decode", type="bf16", seqs=1, new=1, heads=32, kv_heads=8, dim=128, page=16,
             min_len=701, max_len=701, window=0, sink=0),
        # a serving batch with very unequal histories, up to long ones
        dict(name="decode-batch", op="decode", type="fp16", seqs=24, new=1, heads=32, kv_heads=8, dim=128, page=64,
             min_len=300, max_len=65537, window=0, sink=0),
        # the model's own head layout, four tokens per sequence: verification of three drafts
        dict(name="decode-drafts", op="decode", type="bf16", seqs=8, new=4, heads=64, kv_heads=1, dim=512, page=128,
             min_len=2000, max_len=32771, window=0, sink=0),
        # a few short prompts of unequal length, one a single token
        dict(name="prefill-short", op="prefill", type="fp16", seqs=3, min_q=1, max_q=150, hist=0, heads=16, kv_heads=16,
             dim=64, page=16, window=64, sink=4),
        # two long prompts, window over the last 4096 positions
        dict(name="prefill-long", op="prefill", type="bf16", seqs=2, min_q=4099, max_q=8192, hist=0, heads=32,
             kv_heads=8, dim=128, page=64, window=4096, sink=4),
        # the model's head layout and window, a chunk of a longer prompt behind cached history
        dict(name="prefill-chunk", op="prefill", type="bf16", seqs=1, min_q=2049, max_q=2049, hist=3001, heads=64,
             kv_heads=1, dim=512, page=128, window=128, sink=4),
        # one decoding step of a batch: a row per sequence
        dict(name="append-step", op="append", type="bf16", seqs=64, min_q=1, max_q=1, hist=1500, heads=1, dim=512,
             page=128, source="fp32"),
        # a long prompt's keys and values
        dict(name="append-prompt", op="append", type="fp16", seqs=2, min_q=4099, max_q=8192, hist=0, heads=8, dim=128,
             page=64, source="fp32"),
        # the logits of one sequence's draft rows
        dict(name="probs-drafts", op="probs", rows=5, vocab=129280, temperature=0.7),
        # the logits of a whole batch's draft rows
        dict(name="probs-batch", op="probs", rows=320, vocab=129280, temperature=1.0),
        # one sequence's drafts
        dict(name="verify-single", op="verify", seqs=1, drafts=4, vocab=129280),
        # a batch's drafts, some sequences with fewer
        dict(name="verify-batch", op="verify", seqs=64, drafts=5, vocab=129280),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv, group = rng.choice([(8, 4), (8, 8), (16, 1), (1, 64), (4, 3), (2, 16), (1, 7), (5, 5)])
    return kv * group, kv


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "probs", "verify"])
    limit = {key: max(work(c)[key] for c in listed() if c["op"] == op) for key in ("bytes", "flops")}
    while True:
        dim = rng.choice([64, 128, 128, 256, 512])
        page = rng.choice([16, 32, 64, 128, 256])
        heads, kv_heads = _heads(rng)
        window = rng.choice([0, _log_int(rng, 16, 4096)])
        sink = rng.choice([0, rng.randint(1, 64)]) if window else 0
        kind = rng.choice(["bf16", "fp16"])
        if op == "decode":
            lo = _log_int(rng, 1, 60000)
            case = dict(op=op, type=kind, seqs=_log_int(rng, 1, 64), new=rng.choice([1, 1, 1, 2, 3, 5, 8]), heads=heads,
                        kv_heads=kv_heads, dim=dim, page=page, min_len=lo, max_len=_log_int(rng, lo, 65537),
                        window=window, sink=sink)
        elif op == "prefill":
            lo = _log_int(rng, 1, 2000)
            case = dict(op=op, type=kind, seqs=_log_int(rng, 1, 8), min_q=lo, max_q=_log_int(rng, lo, 6000),
                        hist=rng.choice([0, _log_int(rng, 1, 4000)]), heads=heads, kv_heads=kv_heads, dim=dim,
                        page=page, window=window, sink=sink)
        elif op == "append":
            lo = _log_int(rng, 1, 4000)
            case = dict(op=op, type=kind, seqs=_log_int(rng, 1, 64), min_q=lo, max_q=_log_int(rng, lo, 8192),
                        hist=rng.choice([0, _log_int(rng, 1, 4000)]), heads=kv_heads, dim=dim, page=page,
                        source=rng.choice(["fp32", kind]))
        elif op == "probs":
            case = dict(op=op, rows=_log_int(rng, 1, 320), vocab=_log_int(rng, 1000, 200000),
                        temperature=rng.choice([0.0, 1.0, round(rng.uniform(0.3, 1.5), 2)]))
        else:
            case = dict(op=op, seqs=_log_int(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log_int(rng, 1000, 200000))
        w = work(case)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return case


def _lengths(case):
    """Per sequence (new tokens, cache length with them), from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    out = []
    for b in range(case["seqs"]):
        if case["op"] == "decode":
            # the first sequence has the longest history, the others spread over the logarithm
            n = case["new"]
            length = case["max_len"] if b == 0 else _log_int(rng, case["min_len"], case["max_len"])
        else:
            n = case["max_q"] if b == 0 else case["min_q"] if b == 1 else _log_int(rng, case["min_q"], case["max_q"])
            length = n + case["hist"]
        out.append((n, length))
    return out


def _visible(i, window, sink):
    """Number of visible positions of the query at position i."""
    if i < 0:
        return 0
    lo = max(0, i - window + 1) if window else 0
    return i - lo + 1 + min(sink, lo)


def work(case):
    """The bytes and operations of one pass that no implementation can do without."""
    op = case["op"]
    if op == "probs":
        return {"bytes": 8 * case["rows"] * case["vocab"], "flops": 4 * case["rows"] * case["vocab"]}
    if op == "verify":
        # one row of the target's and one of the draft's probabilities per sequence
        return {"bytes": 8 * case["seqs"] * case["vocab"], "flops": 3 * case["seqs"] * case["vocab"]}
    lens = _lengths(case)
    n_tok = sum(n for n, _ in lens)
    if op == "append":
        row = case["heads"] * case["dim"]
        return {"bytes": 2 * n_tok * row * (2 + (4 if case["source"] == "fp32" else 2)), "flops": 0}
    pairs = keys = 0
    for n, length in lens:
        first = max(0, length - n)
        pairs += sum(_visible(i, case["window"], case["sink"]) for i in range(length - n, length))
        lo = max(0, first - case["window"] + 1) if case["window"] else 0
        keys += length - lo + min(case["sink"], lo)
    return {"bytes": 4 * keys * case["kv_heads"] * case["dim"] + 4 * n_tok * case["heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------
# Inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(case, lens, kv_heads, g, seed):
    """Pages in random order, as a server that has run for a while holds them;
    rows past a sequence's length keep what an earlier owner left."""
    page, dt = case["page"], TYPES[case["type"]]
    counts = [-(-length // page) for _, length in lens]
    n_pages = sum(counts) + 3
    width = max(max(counts), 1)
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    shape = (n_pages, page, kv_heads, case["dim"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    return k, v, table.cuda()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = {"case": case}
    if op == "probs":
        # a language model's logits: broad noise and a few likely tokens
        x = torch.randn(case["rows"], case["vocab"], generator=g, device="cuda") * 2.0
        top = torch.randint(case["vocab"], (case["rows"], 8), generator=g, device="cuda")
        x.scatter_add_(1, top, torch.rand(case["rows"], 8, generator=g, device="cuda") * 8 + 4)
        state.update(logits=x, out=torch.empty_like(x))
        return state
    if op == "verify":
        B, G, V = case["seqs"], case["drafts"], case["vocab"]
        base = torch.randn(B, G + 1, V, generator=g, device="cuda") * 2.0
        top = torch.randint(V, (B, G + 1, 8), generator=g, device="cuda")
        base.scatter_add_(2, top, torch.rand(B, G + 1, 8, generator=g, device="cuda") * 8 + 6)
        noise = torch.randn(B, G, V, generator=g, device="cuda") * 0.6
        target = torch.softmax(base, -1)
        draft = torch.softmax(base[:, :G] + noise, -1)
        tokens = torch.multinomial(draft.view(B * G, V), 1, generator=g).view(B, G).int()
        count = torch.randint(max(1, G - 2), G + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        count[0] = G
        state.update(target=target, draft=draft, tokens=tokens, count=count,
                     u_accept=torch.rand(B, G, generator=g, device="cuda"),
                     u_sample=torch.rand(B, generator=g, device="cuda"))
        return state
    lens = _lengths(case)
    n_tok = sum(n for n, _ in lens)
    kv_heads = case["heads"] if op == "append" else case["kv_heads"]
    k, v, table = _cache(case, lens, kv_heads, g, seed)
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    state.update(lens=lens, starts=starts, k=k, v=v, table=table,
                 kv_len=torch.tensor([length for _, length in lens], dtype=torch.int32, device="cuda"),
                 cu_q=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    if op == "append":
        dt = torch.float32 if case["source"] == "fp32" else TYPES[case["type"]]
        shape = (n_tok, kv_heads, case["dim"])
        state["k_new"] = torch.randn(shape, generator=g, device="cuda").to(dt)
        state["v_new"] = torch.randn(shape, generator=g, device="cuda").to(dt)
    else:
        shape = (n_tok, case["heads"], case["dim"])
        if op == "decode":
            shape = (case["seqs"], case["new"]) + shape[1:]
        # queries a little longer than unit normal ones: some keys stand out
        state["q"] = (torch.randn(shape, generator=g, device="cuda") * 1.5).to(TYPES[case["type"]])
        state["out"] = torch.empty_like(state["q"])
    if own:
        import deepseek_v4_flash_gb300 as ds4
        state["cache"] = ds4.KVCache(k, v, table)
        state["attn"] = ds4.Attention(ds4.AttentionDesc(
            n_heads=case["heads"], n_kv_heads=kv_heads, head_dim=case["dim"], dtype=case["type"],
            window=case.get("window", 0), n_sink=case.get("sink", 0), max_seqs=case["seqs"], max_tokens=n_tok))
    return state


# ---------------------------------------------------------------------------
# The plain forms

def _visible_rows(state, b, first, last):
    """Positions of sequence b that queries at first..last see at all, and its
    keys and values there in 32 bits, [kv_heads, positions, dim]."""
    c = state["case"]
    dev = state["k"].device
    lo = max(0, first - c["window"] + 1) if c["window"] else 0
    pos = torch.arange(lo, last + 1, device=dev)
    if lo and c["sink"]:
        pos = torch.cat([torch.arange(min(c["sink"], lo), device=dev), pos])
    page = state["table"][b].long()[pos // c["page"]]
    row = pos % c["page"]
    return pos, state["k"][page, row].float().transpose(0, 1), state["v"][page, row].float().transpose(0, 1)


def _plain_attention(state, b, q, first):
    """q [n, heads, dim] at positions first, first + 1, ... of sequence b."""
    c = state["case"]
    n, heads, dim = q.shape
    kv = c["kv_heads"]
    if first + n <= 0:
        return torch.zeros_like(q)
    pos, k, v = _visible_rows(state, b, max(first, 0), first + n - 1)
    at = torch.arange(first, first + n, device=q.device)[:, None]
    ok = pos[None, :] <= at
    if c["window"]:
        ok = ok & ((pos[None, :] > at - c["window"]) | (pos[None, :] < c["sink"]))
    qg = q.float().view(n, kv, heads // kv, dim).permute(1, 2, 0, 3)
    s = torch.matmul(qg, k[:, None].transpose(2, 3)) * (1.0 / math.sqrt(dim))
    s = torch.where(ok, s, torch.full((), -math.inf, device=s.device))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, None]) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(2, 0, 1, 3).reshape(n, heads, dim).to(q.dtype)


def _run_plain(state):
    c = state["case"]
    op = c["op"]
    if op == "probs":
        x = state["logits"]
        if c["temperature"] == 0:
            top = x.amax(-1, keepdim=True)
            # the lowest index that holds the maximum
            at = torch.where(x == top, torch.arange(x.shape[1], device=x.device), x.shape[1]).amin(-1, keepdim=True)
            return (torch.arange(x.shape[1], device=x.device) == at).float()
        z = (x - x.amax(-1, keepdim=True)) / c["temperature"]
        e = torch.exp(z)
        return e / e.sum(-1, keepdim=True)
    if op == "verify":
        # borders decide whole numbers: 64 bits
        B, G = state["tokens"].shape
        t = state["tokens"].long()[..., None]
        p = state["target"][:, :G].gather(2, t)[..., 0].double()
        q = state["draft"].gather(2, t)[..., 0].double()
        count = state["count"].long()
        ok = (state["u_accept"].double() * q < p) & (torch.arange(G, device=p.device) < count[:, None])
        n = torch.cumprod(ok.long(), 1).sum(1)
        rows = torch.arange(B, device=p.device)
        pr = state["target"][rows, n].double()
        qr = state["draft"][rows, n.clamp(max=G - 1)].double()
        r = torch.where((n < count)[:, None], (pr - qr).clamp(min=0), pr)
        r = torch.where(r.sum(1, keepdim=True) > 0, r, pr)
        cdf = torch.cumsum(r, 1)
        drawn = (cdf <= state["u_sample"].double()[:, None] * cdf[:, -1:]).sum(1)
        i = torch.arange(G + 1, device=p.device)
        padded = torch.cat([state["tokens"].long(), torch.full((B, 1), -1, device=p.device)], 1)
        out = torch.where(i < n[:, None], padded, torch.where(i == n[:, None], drawn[:, None], -1))
        return n.int(), out.int()
    if op == "append":
        ends = state["cu_q"][1:]
        i = torch.arange(state["k_new"].shape[0], dtype=torch.int32, device=ends.device)
        b = torch.searchsorted(ends, i, right=True)
        pos = state["kv_len"][b] - ends[b] + i
        page, row = state["table"][b, pos // c["page"]].long(), pos % c["page"]
        state["k"][page, row] = state["k_new"].to(state["k"].dtype)
        state["v"][page, row] = state["v_new"].to(state["v"].dtype)
        return state["k"], state["v"]
    out = state["out"]
    for b, (n, length) in enumerate(state["lens"]):
        if op == "decode":
            out[b] = _plain_attention(state, b, state["q"][b], length - n)
            continue
        # blocks of queries, so that a block's scores stay small
        a = state["starts"][b]
        for i in range(0, n, 1024):
            e = min(n, i + 1024)
            out[a + i:a + e] = _plain_attention(state, b, state["q"][a + i:a + e], length - n + i)
    return out


def run(state):
    if not own:
        return _run_plain(state)
    import deepseek_v4_flash_gb300 as ds4
    c = state["case"]
    op = c["op"]
    if op == "probs":
        return ds4.token_probs(state["logits"], c["temperature"], out=state["out"])
    if op == "verify":
        return ds4.verify_drafts(state["target"], state["draft"], state["tokens"], state["u_accept"],
                                 state["u_sample"], n_draft=state["count"])
    if op == "append":
        state["attn"].append(state["cache"], state["k_new"], state["v_new"], state["kv_len"], cu_q=state["cu_q"])
        return state["k"], state["v"]
    if op == "decode":
        return state["attn"].decode(state["cache"], state["q"], state["kv_len"], out=state["out"])
    return state["attn"].prefill(state["cache"], state["q"], state["cu_q"], state["kv_len"], out=state["out"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def _exact_attention(case, state):
    """Row by row of the definition, a block of rows at a time, one kv head at
    a time, over a dense copy of each sequence's cache."""
    group = case["heads"] // case["kv_heads"]
    q_all = state["q"].reshape(-1, case["heads"], case["dim"])
    out = torch.zeros(q_all.shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(state["lens"]):
        n_pages = -(-length // case["page"])
        pages = state["table"][b, :n_pages].long()
        for h in range(case["kv_heads"]):
            k = state["k"][pages][:, :, h].reshape(-1, case["dim"])[:length]
            v = state["v"][pages][:, :, h].reshape(-1, case["dim"])[:length]
            for i in range(0, n, 256):
                rows = torch.arange(length - n + i, min(length, length - n + i + 256), device="cuda")
                lo = max(0, int(length - n + i) - case["window"] + 1) if case["window"] else 0
                hi = length - n + i + len(rows)
                if hi <= 0:
                    continue
                cols = torch.tensor(sorted(set(range(min(case["sink"], lo))) | set(range(lo, hi))), device="cuda")
                see = cols.view(1, 1, -1) <= rows.view(-1, 1, 1)
                if case["window"]:
                    near = rows.view(-1, 1, 1) - cols.view(1, 1, -1) < case["window"]
                    see = see & (near | (cols < case["sink"]).view(1, 1, -1))
                qh = q_all[at + i:at + i + len(rows), h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,jd->ngj", qh, k[cols].double()) / math.sqrt(case["dim"])
                s = s.masked_fill(~see, -math.inf)
                w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
                z = w.sum(-1, keepdim=True)
                z[z == 0] = 1.0
                out[at + i:at + i + len(rows), h * group:(h + 1) * group] = \
                    torch.einsum("ngj,jd->ngd", w / z, v[cols].double())
        at += n
    return out.view(state["q"].shape)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "probs":
        x = state["logits"].double()
        if case["temperature"] == 0:
            out = torch.zeros_like(x)
            for r in range(x.shape[0]):
                out[r, int((x[r] == x[r].max()).nonzero()[0])] = 1.0
            return out
        return torch.softmax(x / case["temperature"], -1)
    if op == "verify":
        B, G = state["tokens"].shape
        tokens, count = state["tokens"].tolist(), state["count"].tolist()
        ua, us = state["u_accept"].double().tolist(), state["u_sample"].double().tolist()
        accepted, emitted = [], []
        for b in range(B):
            i = 0
            while i < count[b]:
                t = tokens[b][i]
                if not ua[b][i] * float(state["draft"][b, i, t]) < float(state["target"][b, i, t]):
                    break
                i += 1
            p = state["target"][b, i].double()
            mass = p
            if i < count[b]:
                rest = torch.relu(p - state["draft"][b, i].double())
                if float(rest.sum()) > 0:
                    mass = rest
            ladder = mass.cumsum(0)
            drawn = int(torch.searchsorted(ladder, (us[b] * ladder[-1]).reshape(1), right=True))
            accepted.append(i)
            emitted.append(tokens[b][:i] + [drawn] + [-1] * (G - i))
        return (torch.tensor(accepted, dtype=torch.int32, device="cuda"),
                torch.tensor(emitted, dtype=torch.int32, device="cuda"))
    if op == "append":
        k, v = state["k"].double(), state["v"].double()
        for b, (n, length) in enumerate(state["lens"]):
            for t in range(0, n):
                pos = length - n + t
                # whole runs of rows that share a page
                if t and pos % case["page"]:
                    continue
                run_len = min(n - t, case["page"] - pos % case["page"])
                page, row, a = int(state["table"][b, pos // case["page"]]), pos % case["page"], state["starts"][b] + t
                k[page, row:row + run_len] = state["k_new"][a:a + run_len].double()
                v[page, row:row + run_len] = state["v_new"][a:a + run_len].double()
        return k, v
    if work(case)["flops"] > 4e12:
        return None
    return _exact_attention(case, state)
