"""Attention over a paged cache and the sampling steps, restated in 64 bits
from their formulas, with the error a 16-bit result may carry."""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dt):
    """Largest relative error of one rounding to dt."""
    return torch.finfo(dt).eps / 2


def sees(i, j, window, n_sink):
    return j <= i and (window == 0 or j > i - window or j < n_sink)


def gather(pool, table, b, length):
    """The first `length` positions of sequence b, [length, kv_heads, dim]."""
    page = pool.shape[1]
    if length == 0:
        return pool.new_zeros((0,) + pool.shape[2:])
    pages = table[b, :-(-length // page)].long()
    return pool[pages].reshape((-1,) + pool.shape[2:])[:length]


def attention(q, k, v, first, window, n_sink, scale):
    """q [n, heads, dim] at positions first, first + 1, ...; k, v [len,
    kv_heads, dim]. Returns the result in 64 bits and the error a kernel may
    make that accumulates in 32 bits, rounds each weight to q's type and the
    result once:
      half a step of |out| for the result, half a step of sum(p |v|) for the
      weights, and what the scores' error moves: a score that is off by e
      changes a weight by a factor within 1 +- 2e and so the result by at
      most 4e sum(p |v|) (numerator and denominator). e: dim roundings of
      2^-24 of sum |q k| scale, and 2^-21 for the scale's own rounding, the
      conversion to base 2 and the exponential, relative to the score (at
      least 1). Sums over the cache add 2^-24 per doubling, below 2^-18.
    Rows whose visible keys or values are not finite are left to the caller."""
    n, heads, dim = q.shape
    length, kv = k.shape[0], k.shape[1]
    u = half_step(q.dtype)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if length == 0:
        return out, tol + 1e-30
    i = (first + torch.arange(n, device=q.device))[:, None]
    j = torch.arange(length, device=q.device)[None, :]
    ok = j <= i
    if window:
        ok = ok & ((j > i - window) | (j < n_sink))
    g = heads // kv
    for h in range(kv):
        seen = ok.any(0)
        kk = torch.where(seen[:, None], k[:, h].double(), 0.0)
        vv = torch.where(seen[:, None], v[:, h].double(), 0.0)
        for a in range(h * g, (h + 1) * g):
            qq = q[:, a].double()
            s = torch.where(ok, (qq @ kk.T) * scale, -math.inf)
            size = torch.where(ok, (qq.abs() @ kk.abs().T) * scale, 0.0).amax(1)
            m = s.amax(1, keepdim=True).clamp(min=-1e300)
            p = torch.where(ok, torch.exp(s - m), 0.0)
            z = p.sum(1, keepdim=True)
            p = p / torch.where(z == 0, 1.0, z)
            out[:, a] = p @ vv
            weight = p @ vv.abs()
            e = (dim * 2.0 ** -24 * size + 2.0 ** -21 * size.clamp(min=1.0) + 2.0 ** -18)[:, None]
            tol[:, a] = u * out[:, a].abs() + (u + 4 * e) * weight
    # below the type's normal range a rounding is half of its smallest step
    return out, tol * (1 + u) + torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps


def paged(lens, page, kv_heads, dim, dt, seed, layout="pages", fill=None, spare=2):
    """k, v pools (shuffled pages), block table with -1 where unused. Rows past
    a sequence's length, and spare pages, hold `fill` (NaN by default)."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    n_pages = sum(counts) + spare
    order = torch.randperm(n_pages, generator=g)
    width = max(counts + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    pools = []
    fill = math.nan if fill is None else fill
    if layout == "pages":
        pools = [torch.full((n_pages, page, kv_heads, dim), fill, dtype=dt) for _ in range(2)]
    elif layout == "heads":  # [page][head][row][dim]
        pools = [torch.full((n_pages, kv_heads, page, dim), fill, dtype=dt).transpose(1, 2) for _ in range(2)]
    else:  # keys and values of a row next to each other
        both = torch.full((n_pages, page, 2, kv_heads, dim), fill, dtype=dt)
        pools = [both[:, :, 0], both[:, :, 1]]
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c].int()
        for p in pools:
            x = torch.randn(lens[b], kv_heads, dim, generator=g).to(dt)
            for i in range(c):
                e = min(lens[b], (i + 1) * page)
                p[order[at + i], :e - i * page] = x[i * page:e]
        at += c
    return pools[0], pools[1], table


def to_cuda(k, v):
    """Device copies with the same strides."""
    out = []
    base = {}
    for t in (k, v):
        s = t.untyped_storage()
        if s.data_ptr() not in base:
            base[s.data_ptr()] = torch.empty(0, dtype=t.dtype).set_(s).cuda()
        out.append(base[s.data_ptr()].as_strided(t.shape, t.stride(), t.storage_offset()))
    return out
