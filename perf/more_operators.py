"""Operators of a serving step for many requests at once, as cases to measure.

Projections carry a request's low-rank adapter beside the shared matrix
(``adapt``), the new queries and keys are rotated by their positions on the way
into the paged cache (``rotate``), and a batch whose sequences begin with the
same positions attends to those once (``shared``).

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, 64 for the angles of far positions), or, with ``own`` set, through the
package's public entry points. ``exact`` evaluates the definition in 64 bits,
written apart from the plain form.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one user's next token with the model's own head layout: the last 64 of 512 elements turn, pairs of neighbours
        dict(name="rotate-single", op="rotate", type="bf16", source="fp32", seqs=1, min_q=1, max_q=1, hist=700, heads=64,
             kv_heads=1, dim=512, page=128, rot=64, offset=448, pairs="neighbours", base=10000.0),
        # one decoding step of a batch, far into long histories
        dict(name="rotate-step", op="rotate", type="bf16", source="fp32", seqs=64, min_q=1, max_q=1, hist=131071,
             heads=32, kv_heads=8, dim=128, page=64, rot=128, offset=0, pairs="halves", base=500000.0),
        # the prompts of two users
        dict(name="rotate-prompt", op="rotate", type="fp16", source="fp32", seqs=2, min_q=4099, max_q=8192, hist=0,
             heads=32, kv_heads=8, dim=128, page=64, rot=128, offset=0, pairs="halves", base=10000.0),
        # chunks of longer prompts, projections already in the cache's type, a quarter of each head turns
        dict(name="rotate-chunk", op="rotate", type="bf16", source="bf16", seqs=5, min_q=1, max_q=1023, hist=3001,
             heads=16, kv_heads=16, dim=64, page=16, rot=16, offset=0, pairs="halves", base=10000.0),
        # a few users of one assistant, its instructions before them: latency counts
        dict(name="shared-few", op="shared", type="bf16", groups="8", new=1, heads=32, kv_heads=8, dim=128, page=16,
             prefix=1501, min_own=1, max_own=200),
        # a full batch behind one long document
        dict(name="shared-batch", op="shared", type="fp16", groups="64", new=1, heads=32, kv_heads=8, dim=128, page=64,
             prefix=32771, min_own=100, max_own=2000),
        # drafts checked with the model's own head layout
        dict(name="shared-drafts", op="shared", type="bf16", groups="16", new=4, heads=64, kv_heads=1, dim=512,
             page=128, prefix=16384, min_own=50, max_own=4000),
        # three assistants and a user alone in one batch
        dict(name="shared-groups", op="shared", type="bf16", groups="20,1,7,12", new=2, heads=16, kv_heads=4, dim=64,
             page=32, prefix=6000, min_own=2, max_own=1000),
        # one request's next token
        dict(name="adapt-single", op="adapt", type="bf16", source="fp32", seqs=1, min_q=1, max_q=1, slots=4, none=0,
             min_rank=16, max_rank=16, n_in=4096, n_out=4096),
        # a decoding step of many requests, adapters of unequal rank, some without
        dict(name="adapt-step", op="adapt", type="bf16", source="fp32", seqs=64, min_q=1, max_q=1, slots=48, none=8,
             min_rank=8, max_rank=64, n_in=4096, n_out=4096),
        # prompts of a few requests
        dict(name="adapt-prompt", op="adapt", type="bf16", source="fp32", seqs=4, min_q=1000, max_q=3001, slots=4,
             none=0, min_rank=64, max_rank=64, n_in=4096, n_out=4096),
        # chunks of many short prompts into the attention's output of eight key-value heads
        dict(name="adapt-chunk", op="adapt", type="fp16", source="fp16", seqs=19, min_q=3, max_q=150, slots=12, none=2,
             min_rank=5, max_rank=128, n_in=4096, n_out=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "shared", "shared", "adapt", "adapt"])
    limit = {key: max(work(c)[key] for c in listed() if c["op"] == op) for key in ("bytes", "flops")}
    while True:
        dim = rng.choice([64, 128, 128, 256, 512])
        kv, group = rng.choice([(8, 4), (8, 8), (16, 1), (1, 64), (4, 3), (2, 16), (1, 7), (5, 5)])
        kind = rng.choice(["bf16", "fp16"])
        page = rng.choice([16, 32, 64, 128, 256])
        if op == "rotate":
            lo = _log_int(rng, 1, 4000)
            rot = rng.choice([16, 32, dim // 2, dim // 4 * 3 // 16 * 16, dim])
            case = dict(op=op, type=kind, source=rng.choice(["fp32", kind]), seqs=_log_int(rng, 1, 64), min_q=lo,
                        max_q=_log_int(rng, lo, 8192), hist=rng.choice([0, _log_int(rng, 1, 200000)]),
                        heads=kv * group, kv_heads=kv, dim=dim, page=page, rot=rot,
                        offset=rng.choice([0, dim - rot]), pairs=rng.choice(["halves", "neighbours"]),
                        base=rng.choice([10000.0, 500000.0, 1000000.0]))
        elif op == "shared":
            groups = [_log_int(rng, 1, 64) for _ in range(rng.choice([1, 1, 2, 3, 6]))]
            own_lo = _log_int(rng, 1, 1000)
            case = dict(op=op, type=kind, groups=",".join(map(str, groups)), new=rng.choice([1, 1, 1, 2, 3, 5]),
                        heads=kv * group, kv_heads=kv, dim=dim, page=page, prefix=_log_int(rng, 1, 40000),
                        min_own=own_lo, max_own=_log_int(rng, own_lo, 4000))
            case["min_own"] = max(case["min_own"], case["new"])
            case["max_own"] = max(case["max_own"], case["min_own"])
        else:
            lo = _log_int(rng, 1, 1500)
            rank = _log_int(rng, 1, 128)
            case = dict(op=op, type=kind, source=rng.choice(["fp32", "fp32", kind]), seqs=_log_int(rng, 1, 64),
                        min_q=lo, max_q=_log_int(rng, lo, 3000), slots=_log_int(rng, 1, 64), none=rng.choice([0, 0, 1, 5]),
                        min_rank=rank, max_rank=_log_int(rng, rank, 128),
                        n_in=32 * _log_int(rng, 8, 256), n_out=_log_int(rng, 256, 8192))
        w = work(case)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return case


def _fixed(case):
    """A random.Random that depends on the case alone."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _new_tokens(case):
    """New tokens of each sequence."""
    rng = _fixed(case)
    out = []
    for b in range(case["seqs"]):
        out.append(case["max_q"] if b == 0 else case["min_q"] if b == 1 else _log_int(rng, case["min_q"], case["max_q"]))
    return out


def _slots(case):
    """The adapter of each sequence (-1: none) and the rank of each adapter."""
    rng = _fixed(case)
    ranks = [case["max_rank"] if s == 0 else _log_int(rng, case["min_rank"], case["max_rank"]) for s in range(case["slots"])]
    of = list(range(case["slots"])) * (case["seqs"] // case["slots"] + 1)
    rng.shuffle(of)
    of = of[:case["seqs"]]
    for b in rng.sample(range(1, case["seqs"]), min(case["none"], case["seqs"] - 1)):
        of[b] = -1
    return of, ranks


def _shared_lengths(case):
    """Per group (first sequence, end, shared positions) and the length of each sequence."""
    rng = _fixed(case)
    groups, lens = [], []
    for i, n in enumerate(int(x) for x in case["groups"].split(",")):
        prefix = case["prefix"] if i == 0 else _log_int(rng, max(1, case["prefix"] // 8), case["prefix"])
        groups.append((len(lens), len(lens) + n, prefix))
        for b in range(n):
            mine = case["max_own"] if b == 0 else _log_int(rng, case["min_own"], case["max_own"])
            lens.append(prefix + mine)
    return groups, lens


def work(case):
    """The bytes and operations of one pass that no implementation can do without."""
    op = case["op"]
    if op == "rotate":
        n, src = sum(_new_tokens(case)), 4 if case["source"] == "fp32" else 2
        rows = case["heads"] + 2 * case["kv_heads"]
        return {"bytes": n * rows * case["dim"] * (src + 2),
                "flops": 3 * n * (case["heads"] + case["kv_heads"]) * case["rot"]}
    if op == "shared":
        groups, lens = _shared_lengths(case)
        new = case["new"]
        keys = sum(s for _, _, s in groups) + sum(lens[b] - s for a, e, s in groups for b in range(a, e))
        pairs = sum(new * n - new * (new - 1) // 2 for n in lens)
        return {"bytes": 4 * keys * case["kv_heads"] * case["dim"] + 4 * len(lens) * new * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    tokens, (of, ranks) = _new_tokens(case), _slots(case)
    src = 4 if case["source"] == "fp32" else 2
    n = sum(tokens)
    read = sum(t for t, s in zip(tokens, of) if s >= 0)
    r = sum(t * ranks[s] for t, s in zip(tokens, of) if s >= 0)
    there = sum(ranks[s] for s in set(of) if s >= 0)
    return {"bytes": read * case["n_in"] * src + 8 * n * case["n_out"] + 2 * there * (case["n_in"] + case["n_out"]),
            "flops": 2 * r * (case["n_in"] + case["n_out"])}


# ---------------------------------------------------------------------------
# Inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(case, n_pages, g):
    shape = (n_pages, case["page"], case["kv_heads"], case["dim"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=TYPES[case["type"]]) for _ in range(2)]


def _prepare_rotate(case, seed, g, state):
    tokens = _new_tokens(case)
    n, page = sum(tokens), case["page"]
    lens = [t + case["hist"] for t in tokens]
    counts = [-(-x // page) for x in lens]
    old = case["hist"] // page  # pages before them are not touched: they are left out of the pool
    order = list(range(sum(counts) - old * len(lens) + 3))
    random.Random(seed).shuffle(order)  # pages in random order, as a server that has run for a while holds them
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, old:c] = torch.tensor(order[at:at + c - old], dtype=torch.int32)
        at += c - old
    starts = [0]
    for t in tokens:
        starts.append(starts[-1] + t)
    state["k"], state["v"] = _pool(case, len(order), g)
    src = TYPES[case["source"]]
    i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float32)
    state.update(
        starts=starts, lens=lens, table=table.cuda(),
        kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        cu_q=torch.tensor(starts, dtype=torch.int32, device="cuda"),
        inv_freq=1.0 / case["base"] ** (i / case["rot"]),
        q_new=torch.randn(n, case["heads"], case["dim"], generator=g, device="cuda").to(src),
        k_new=torch.randn(n, case["kv_heads"], case["dim"], generator=g, device="cuda").to(src),
        v_new=torch.randn(n, case["kv_heads"], case["dim"], generator=g, device="cuda").to(src),
        q_out=torch.empty(n, case["heads"], case["dim"], device="cuda", dtype=TYPES[case["type"]]))
    if own:
        import deepseek_v4_flash_gb300 as ds4
        state["cache"] = ds4.KVCache(state["k"], state["v"], state["table"])
        state["rope"] = ds4.Rope(state["inv_freq"], offset=case["offset"], interleaved=case["pairs"] == "neighbours")
        state["attn"] = ds4.Attention(ds4.AttentionDesc(
            n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype=case["type"],
            max_seqs=len(lens), max_tokens=n))


def _prepare_shared(case, seed, g, state):
    groups, lens = _shared_lengths(case)
    page = case["page"]
    width = -(-max(lens) // page)
    total = sum(s // page for _, _, s in groups) + \
        sum(-(-lens[b] // page) - s // page for a, e, s in groups for b in range(a, e))
    order = list(range(total + 3))
    random.Random(seed).shuffle(order)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    k, v = _pool(case, len(order), g)
    for a, e, s in groups:
        whole, rest = s // page, s % page
        table[a:e, :whole] = torch.tensor(order[at:at + whole], dtype=torch.int32)
        at += whole
        for b in range(a, e):
            c = -(-lens[b] // page) - whole
            table[b, whole:whole + c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
            if rest and b > a:  # the page in which the shared positions end: every sequence has its copy
                for t in (k, v):
                    t[int(table[b, whole]), :rest] = t[int(table[a, whole]), :rest]
    n_tok = len(lens) * case["new"]
    state["q"] = (torch.randn(len(lens), case["new"], case["heads"], case["dim"], generator=g, device="cuda") * 1.5).to(
        TYPES[case["type"]])
    state.update(
        k=k, v=v, groups=groups, lens=lens, table=table.cuda(), out=torch.empty_like(state["q"]),
        kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        shared_len=torch.tensor([s for _, _, s in groups], dtype=torch.int32, device="cuda"),
        group_start=torch.tensor([a for a, _, _ in groups] + [len(lens)], dtype=torch.int32, device="cuda"))
    if own:
        import deepseek_v4_flash_gb300 as ds4
        state["cache"] = ds4.KVCache(k, v, state["table"])
        state["attn"] = ds4.Attention(ds4.AttentionDesc(
            n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype=case["type"],
            max_seqs=len(lens), max_tokens=n_tok, max_shared_tokens=n_tok))


def _prepare_adapt(case, seed, g, state):
    tokens, (of, ranks) = _new_tokens(case), _slots(case)
    n, dt = sum(tokens), TYPES[case["type"]]
    n_in, n_out = case["n_in"], case["n_out"]
    runs, at = [], 0
    for t, s in zip(tokens, of):
        runs.append((at, at + t, s))
        at += t
    a = [(torch.randn(r, n_in, generator=g, device="cuda") / math.sqrt(n_in)).to(dt) for r in ranks]
    b = [(torch.randn(n_out, r, generator=g, device="cuda") * 0.3).to(dt) for r in ranks]
    scales = [2.0 * 16 / r for r in ranks]
    state.update(
        runs=runs, a=a, b=b, scales=scales,
        slots=torch.tensor([s for t, s in zip(tokens, of) for _ in range(t)], dtype=torch.int32, device="cuda"),
        x=torch.randn(n, n_in, generator=g, device="cuda").to(TYPES[case["source"]]),
        base=torch.randn(n, n_out, generator=g, device="cuda"), y=torch.empty(n, n_out, device="cuda"))
    if own:
        import deepseek_v4_flash_gb300 as ds4
        ad = ds4.Adapters(n_out, n_in, n_slots=len(ranks), max_rank=max(ranks), dtype=case["type"], max_tokens=n)
        for i in range(len(ranks)):
            ad.set(i, a[i], b[i], scales[i])
        state["adapters"] = ad


def prepare(case, seed):
    state = {"case": case}
    {"rotate": _prepare_rotate, "shared": _prepare_shared, "adapt": _prepare_adapt}[case["op"]](
        case, seed, _generator(seed), state)
    return state


# ---------------------------------------------------------------------------
# The plain forms

def _rotate(x, c, cos, sin, dt):
    """x [n, heads, dim] in 32 bits, cos and sin [n, 1, rot / 2]; rounded to dt."""
    o, r = c["offset"], c["rot"]
    part = x[..., o:o + r]
    if c["pairs"] == "halves":
        a, b = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :o], turned, x[..., o + r:]], -1).to(dt)


def _plain_rotate(state):
    c = state["case"]
    ends = state["cu_q"][1:]
    i = torch.arange(state["k_new"].shape[0], dtype=torch.int32, device=ends.device)
    b = torch.searchsorted(ends, i, right=True)
    pos = state["kv_len"][b] - ends[b] + i
    angle = pos.double()[:, None, None] * state["inv_freq"].double()  # far positions: 64 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    page, row = state["table"][b, pos // c["page"]].long(), pos % c["page"]
    dt = state["k"].dtype
    state["q_out"].copy_(_rotate(state["q_new"].float(), c, cos, sin, dt))
    state["k"][page, row] = _rotate(state["k_new"].float(), c, cos, sin, dt)
    state["v"][page, row] = state["v_new"].to(dt)
    return state["q_out"], state["k"], state["v"]


def _positions(state, b, first, end):
    """Keys and values of sequence b at positions first .. end - 1 in 32 bits, [kv_heads, positions, dim]."""
    c = state["case"]
    pos = torch.arange(first, end, device=state["k"].device)
    page, row = state["table"][b, pos // c["page"]].long(), pos % c["page"]
    return state["k"][page, row].float().transpose(0, 1), state["v"][page, row].float().transpose(0, 1)


def _plain_shared(state):
    c = state["case"]
    kv, group, dim, new = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["new"]
    scale = 1.0 / math.sqrt(dim)
    for a, e, s in state["groups"]:
        n = e - a
        # rows of a key-value head: [kv, sequence, new, group, dim]
        q = state["q"][a:e].float().view(n, new, kv, group, dim).permute(2, 0, 1, 3, 4) * scale
        k, v = _positions(state, a, 0, s)
        far = torch.matmul(q.reshape(kv, -1, dim), k.transpose(1, 2)).view(kv, n, new, group, s)
        top = far.amax(-1)
        far = torch.exp(far - top[..., None])
        total = far.sum(-1)
        o = torch.matmul(far.view(kv, -1, s), v).view(kv, n, new, group, dim)
        del far
        for b in range(a, e):
            length = state["lens"][b]
            kb, vb = _positions(state, b, s, length)
            near = torch.matmul(q[:, b - a].reshape(kv, -1, dim), kb.transpose(1, 2)).view(kv, new, group, length - s)
            at = torch.arange(length - new, length, device=q.device)[:, None, None]
            near = torch.where(torch.arange(s, length, device=q.device) <= at, near, -math.inf)
            m = torch.maximum(near.amax(-1), top[:, b - a])
            w = torch.exp(near - m[..., None])
            f = torch.exp(top[:, b - a] - m)
            z = total[:, b - a] * f + w.sum(-1)
            y = torch.matmul(w.view(kv, -1, length - s), vb).view(kv, new, group, dim)
            y = (o[:, b - a] * f[..., None] + y) / z[..., None]
            state["out"][b] = y.permute(1, 0, 2, 3).reshape(new, kv * group, dim)
    return state["out"]


def _plain_adapt(state):
    y = state["y"]
    y.copy_(state["base"])
    for i, e, s in state["runs"]:
        if s >= 0:
            h = state["x"][i:e].float() @ state["a"][s].float().T
            y[i:e] += (h * state["scales"][s]) @ state["b"][s].float().T
    return y


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rotate": _plain_rotate, "shared": _plain_shared, "adapt": _plain_adapt}[op](state)
    if op == "rotate":
        q = state["attn"].append(state["cache"], state["k_new"], state["v_new"], state["kv_len"], cu_q=state["cu_q"],
                                 rope=state["rope"], q=state["q_new"], q_out=state["q_out"])
        return q, state["k"], state["v"]
    if op == "shared":
        return state["attn"].decode(state["cache"], state["q"], state["kv_len"], out=state["out"],
                                    shared_len=state["shared_len"], group_start=state["group_start"])
    return state["adapters"].forward(state["x"], state["slots"], state["y"], base=state["base"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def _exact_rotate(case, state):
    def turned(x, first):
        """Rows x [n, heads, dim] of positions first, first + 1, ... as complex numbers times exp(i angle)."""
        x = x.double()
        at = torch.arange(first, first + x.shape[0], device="cuda", dtype=torch.float64)
        angle = torch.outer(at, state["inv_freq"].double())
        o, half = case["offset"], case["rot"] // 2
        j = torch.arange(half, device="cuda")
        ia, ib = (o + j, o + half + j) if case["pairs"] == "halves" else (o + 2 * j, o + 2 * j + 1)
        z = torch.complex(x[:, :, ia], x[:, :, ib]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        x[:, :, ia], x[:, :, ib] = z.real, z.imag
        return x
    k, v = state["k"].double(), state["v"].double()
    qs = []
    for b, length in enumerate(state["lens"]):
        i, e = state["starts"][b], state["starts"][b + 1]
        first = length - (e - i)
        qs.append(turned(state["q_new"][i:e], first))
        kk = turned(state["k_new"][i:e], first)
        t = 0
        while t < e - i:
            # whole runs of rows that share a page
            p, r = divmod(first + t, case["page"])
            m = min(e - i - t, case["page"] - r)
            at = int(state["table"][b, p])
            k[at, r:r + m] = kk[t:t + m]
            v[at, r:r + m] = state["v_new"][i + t:i + t + m].double()
            t += m
    return torch.cat(qs), k, v


def _exact_shared(case, state):
    """Every sequence by itself over a dense copy of its whole cache."""
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(state["lens"]):
        pages = state["table"][b, :-(-length // case["page"])].long()
        k = state["k"][pages].flatten(0, 1)[:length].double()
        v = state["v"][pages].flatten(0, 1)[:length].double()
        q = state["q"][b].double().unflatten(1, (case["kv_heads"], group))
        s = torch.einsum("nhgd,jhd->nhgj", q, k) / math.sqrt(case["dim"])
        for i in range(case["new"]):
            s[i, :, :, length - case["new"] + i + 1:] = -math.inf
        out[b] = torch.einsum("nhgj,jhd->nhgd", torch.softmax(s, -1), v).flatten(1, 2)
    return out


def _exact_adapt(case, state):
    y = state["base"].double()
    slots = state["slots"].tolist()
    for s in sorted(set(slots) - {-1}):
        rows = torch.tensor([t for t, x in enumerate(slots) if x == s], device="cuda")
        delta = state["scales"][s] * torch.linalg.multi_dot(
            [state["x"][rows].double(), state["a"][s].double().T, state["b"][s].double().T])
        y.index_add_(0, rows, delta)
    return y


def exact(case, seed):
    state = prepare(case, seed)
    if work(case)["flops"] > 4e12:
        return None
    return {"rotate": _exact_rotate, "shared": _exact_shared, "adapt": _exact_adapt}[case["op"]](case, state)
