"""The attention operators (ds4moe_kv_append, ds4moe_attn_decode,
ds4moe_attn_prefill) on the GPU against their formulas in 64 bits."""
import math

import pytest
import torch

from tests.attn_ref import DTYPES, attention, gather, paged, to_cuda

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


def _handle(ds4, kind, heads, kv, dim, window, sink, n_seq, n_tok, scale=None):
    return ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, window, sink, scale, max(n_seq, 1), max(n_tok, 1)))


def _check(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values are not finite"
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {got.numel()} off, worst by {float(over.max())} " \
                              f"(error {float((got - ref).abs().max())})"


def _run_decode(kind, heads, kv, dim, page, window, sink, new, lens, seed=0, layout="pages", qscale=1.5, scale=None):
    ds4 = _ds4()
    dt = DTYPES[kind]
    k, v, table = paged(lens, page, kv, dim, dt, seed, layout)
    kd, vd = to_cuda(k, v)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), new, heads, dim, generator=g) * qscale).to(dt).cuda()
    at = _handle(ds4, kind, heads, kv, dim, window, sink, len(lens), len(lens) * new, scale)
    cache = ds4.KVCache(kd, vd, table.cuda())
    out = at.decode(cache, q, torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert at.device_error() == 0
    for b, n in enumerate(lens):
        ref, tol = attention(q[b], gather(kd, table, b, n), gather(vd, table, b, n), n - new, window, sink,
                             scale or dim ** -0.5)
        _check(out[b], ref, tol, f"sequence {b} of length {n}")
    again = at.decode(cache, q, torch.tensor(lens, dtype=torch.int32).cuda())
    assert torch.equal(out, again), "two calls differ"
    at.close()


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1021]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,dim", [(8, 8, 64), (32, 4, 128), (6, 2, 64), (7, 1, 128), (16, 1, 128),
                                          (8, 2, 256), (64, 1, 512), (5, 5, 512), (128, 1, 64), (40, 2, 128)])
def test_decode_one_token(kind, heads, kv, dim):
    _run_decode(kind, heads, kv, dim, 16, 0, 0, 1, LENS, seed=heads + dim)


@pytest.mark.parametrize("heads,kv,dim,new", [(8, 8, 64, 2), (8, 2, 128, 3), (8, 2, 128, 5), (64, 1, 512, 4),
                                              (64, 1, 512, 3), (12, 4, 256, 16), (6, 2, 64, 7), (100, 1, 128, 2)])
def test_decode_several_tokens(heads, kv, dim, new):
    """Drafted tokens, among them sequences shorter than the new tokens."""
    _run_decode("bf16", heads, kv, dim, 32, 0, 0, new, LENS, seed=new)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,new", [(64, 1, 2), (64, 1, 5), (64, 1, 16), (128, 1, 1), (128, 1, 5), (16, 2, 16), (20, 4, 13)])
def test_decode_pairs_of_row_tiles(kind, heads, kv, new):
    """Dimension 512: one row tile, an even and an odd number of them, tiles
    that the group of heads does not fill, over whole and windowed caches."""
    _run_decode(kind, heads, kv, 512, 64, 0, 0, new, LENS + [5000], seed=new)
    _run_decode(kind, heads, kv, 512, 16, 150, 20, new, LENS + [2000], seed=new + 1)


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (16, 0), (100, 4), (128, 4), (129, 40), (300, 200), (5000, 7)])
@pytest.mark.parametrize("heads,kv,dim,new", [(8, 2, 128, 1), (4, 4, 64, 3), (64, 1, 512, 2), (8, 1, 256, 4)])
def test_decode_window(window, sink, heads, kv, dim, new):
    _run_decode("bf16", heads, kv, dim, 16, window, sink, new, LENS + [2050], seed=window)


@pytest.mark.parametrize("page", [16, 48, 64, 128, 256, 1024])
def test_decode_pages(page):
    """Pages of every size, also one that is not a power of two."""
    for heads, kv, dim, new in [(8, 2, 128, 1), (64, 1, 512, 1), (32, 2, 64, 4)]:
        _run_decode("bf16", heads, kv, dim, page, 0, 0, new, [1, page - 1, page, page + 1, 2 * page + 3, 500], seed=page)


@pytest.mark.parametrize("layout", ["heads", "fused"])
def test_decode_layouts(layout):
    for heads, kv, dim, new in [(8, 2, 128, 1), (64, 2, 512, 1), (12, 4, 64, 9)]:
        _run_decode("fp16", heads, kv, dim, 32, 70, 3, new, [5, 77, 400], seed=3, layout=layout)


def test_decode_long():
    """One long sequence (split over the cache) and a batch of unequal ones."""
    for heads, kv, dim, new in [(32, 8, 128, 1), (64, 1, 512, 4), (8, 8, 64, 1), (16, 2, 256, 2)]:
        _run_decode("bf16", heads, kv, dim, 64, 0, 0, new, [30011], seed=7)
        _run_decode("fp16", heads, kv, dim, 64, 0, 0, new, [9001, 3, 0, 12345, 1, 640, 64, 128, 4097], seed=8)


def test_many_sequences():
    """More sequences than a warp has lanes, empty ones among them."""
    lens = [(37 * i) % 300 for i in range(70)]
    for heads, kv, dim, new in [(8, 2, 128, 1), (64, 1, 512, 1), (8, 1, 256, 3), (40, 2, 64, 2)]:
        _run_decode("bf16", heads, kv, dim, 16, 0, 0, new, lens, seed=11)
    runs = [((7 * i) % 11, (13 * i) % 50) for i in range(70)]
    for heads, kv, dim in [(4, 2, 128), (8, 1, 256), (64, 1, 512)]:
        _run_prefill("bf16", heads, kv, dim, 16, 20, 3, runs, seed=12)


def test_many_row_groups():
    """Prompts whose row groups every block no longer walks through itself:
    one of 600 groups, and two short ones behind it."""
    _run_prefill("bf16", 64, 1, 64, 32, 64, 4, [(2400, 0), (3, 2), (0, 9), (70, 100)], seed=4)
    _run_prefill("fp16", 128, 1, 512, 32, 64, 4, [(1030, 7), (5, 0)], seed=5)


@pytest.mark.parametrize("qscale", [0.0, 30.0])
def test_decode_flat_and_peaked_scores(qscale):
    """Equal weights, and scores hundreds apart (the running maximum moves)."""
    for heads, kv, dim, new in [(8, 2, 128, 1), (64, 1, 512, 2), (64, 2, 64, 2)]:
        for kind in DTYPES:
            _run_decode(kind, heads, kv, dim, 64, 0, 0, new, [2, 700, 3000], seed=9, qscale=qscale)


def test_decode_rising_scores():
    """Scores that grow along the cache: the maximum is at the last position,
    and early weights vanish against it; and scores that fall."""
    ds4 = _ds4()
    for heads, kv, dim in [(8, 2, 128), (64, 1, 512), (64, 1, 128)]:
        for sign in (1, -1):
            for kind, dt in DTYPES.items():
                n = 2000
                k, v, table = paged([n], 64, kv, dim, dt, 3)
                for pos in range(n):
                    k[table[0, pos // 64], pos % 64] = 0
                    k[table[0, pos // 64], pos % 64, :, 0] = sign * 0.1 * pos
                kd, vd = to_cuda(k, v)
                q = torch.zeros(1, 1, heads, dim, dtype=dt)
                q[..., 0] = 1.0
                q = q.cuda()
                at = _handle(ds4, kind, heads, kv, dim, 0, 0, 1, 1, scale=1.0)
                out = at.decode(ds4.KVCache(kd, vd, table.cuda()), q, torch.tensor([n], dtype=torch.int32).cuda())
                ref, tol = attention(q[0], gather(kd, table, 0, n), gather(vd, table, 0, n), n - 1, 0, 0, 1.0)
                _check(out[0], ref, tol, f"{kind} {heads}/{kv}x{dim} sign {sign}")


def _run_prefill(kind, heads, kv, dim, page, window, sink, runs, seed=0, layout="pages", qkv=False):
    """runs: (new tokens, cached positions before them) of each sequence."""
    ds4 = _ds4()
    dt = DTYPES[kind]
    lens = [n + h for n, h in runs]
    T = sum(n for n, _ in runs)
    k, v, table = paged(lens, page, kv, dim, dt, seed, layout)
    kd, vd = to_cuda(k, v)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(T, heads, dim, generator=g) * 1.5).to(dt).cuda()
    out = torch.full_like(q, math.nan)
    if qkv:  # q and out as slices of wider rows
        wide = torch.zeros(T, heads + 2 * kv, dim, dtype=dt, device="cuda")
        wide[:, :heads] = q
        q = wide[:, :heads]
        out = torch.full_like(wide, math.nan)[:, kv:kv + heads]
    cu = [0]
    for n, _ in runs:
        cu.append(cu[-1] + n)
    at = _handle(ds4, kind, heads, kv, dim, window, sink, len(runs), T)
    cache = ds4.KVCache(kd, vd, table.cuda())
    cu_d, len_d = torch.tensor(cu, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    at.prefill(cache, q, cu_d, len_d, out=out)
    torch.cuda.synchronize()
    assert at.device_error() == 0
    for b, (n, h) in enumerate(runs):
        if n == 0:
            continue
        ref, tol = attention(q[cu[b]:cu[b + 1]], gather(kd, table, b, n + h), gather(vd, table, b, n + h), h, window,
                             sink, dim ** -0.5)
        _check(out[cu[b]:cu[b + 1]], ref, tol, f"run {b}: {n} tokens after {h}")
    again = at.prefill(cache, q, cu_d, len_d)
    assert torch.equal(out, again), "two calls differ"
    at.close()


RUNS = [(0, 0), (1, 0), (17, 0), (0, 40), (130, 0), (1, 500), (64, 333), (257, 5), (128, 128)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,dim", [(4, 4, 64), (8, 2, 128), (6, 2, 64), (7, 1, 128), (4, 1, 256), (64, 1, 512),
                                          (3, 3, 512), (128, 1, 64)])
def test_prefill_ragged(kind, heads, kv, dim):
    _run_prefill(kind, heads, kv, dim, 16, 0, 0, RUNS, seed=heads)


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 3), (16, 0), (64, 4), (128, 4), (129, 17), (250, 300), (4096, 4)])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (2, 2, 64), (4, 1, 256), (64, 1, 512)])
def test_prefill_window(window, sink, heads, kv, dim):
    _run_prefill("bf16", heads, kv, dim, 32, window, sink, RUNS + [(300, 900)], seed=window + sink)


@pytest.mark.parametrize("window", [200, 500, 700, 960])
@pytest.mark.parametrize("heads,kv,dim", [(32, 1, 128), (16, 4, 64), (8, 1, 256), (64, 1, 512)])
def test_windows_of_some_tiles(window, heads, kv, dim):
    """Windows of two to eight tiles, few and many sequences: items that stay
    in one block, and items that are split."""
    _run_decode("bf16", heads, kv, dim, 16, window, 4, 5, [2500], seed=window)
    _run_decode("fp16", heads, kv, dim, 64, window, 4, 3, [(311 * i) % 1600 for i in range(60)], seed=window)
    _run_prefill("bf16", heads, kv, dim, 64, window, 4, [(700, 1000)], seed=window)
    _run_prefill("fp16", heads, kv, dim, 32, window, 4, [((29 * i) % 90, (401 * i) % 1500) for i in range(40)], seed=window)


def test_prefill_long():
    for heads, kv, dim, window in [(4, 1, 128, 0), (4, 2, 128, 1000), (2, 2, 64, 0), (16, 1, 512, 128), (2, 1, 256, 0)]:
        _run_prefill("bf16", heads, kv, dim, 64, window, 4 if window else 0, [(2113, 0), (5, 4000), (700, 2000)], seed=2)


def test_prefill_strides_and_layouts():
    for layout in ("pages", "heads", "fused"):
        for heads, kv, dim in [(8, 2, 128), (4, 4, 64), (64, 1, 512)]:
            _run_prefill("bf16", heads, kv, dim, 64, 100, 5, [(33, 0), (200, 71)], seed=5, layout=layout, qkv=True)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (4, 4, 64), (64, 1, 512), (4, 1, 256)])
def test_unseen_positions_do_not_leak(bad, heads, kv, dim):
    """Infinities and NaN at positions that a row does not see: later
    positions of a prefill, and positions between the first ones and the
    window. (Rows past the length hold NaN in every test here.)"""
    ds4 = _ds4()
    n, window, sink = 300, 50, 4
    k, v, table = paged([n], 16, kv, dim, torch.bfloat16, 11)
    kc, vc = to_cuda(k, v)  # a clean copy for the formula
    for pos in (100, 101, 250):
        k[table[0, pos // 16], pos % 16] = bad
        v[table[0, pos // 16], pos % 16] = bad
    kd, vd = to_cuda(k, v)
    cache = ds4.KVCache(kd, vd, table.cuda())
    g = torch.Generator().manual_seed(4)
    q = torch.randn(n, heads, dim, generator=g).bfloat16().cuda()
    at = _handle(ds4, "bf16", heads, kv, dim, window, sink, 1, n)
    out = at.prefill(cache, q, torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    ref, tol = attention(q, gather(kc, table, 0, n), gather(vc, table, 0, n), 0, window, sink, dim ** -0.5)
    touched = torch.zeros(n, dtype=torch.bool)
    for pos in (100, 101, 250):
        touched[pos:pos + window] = True
    _check(out[~touched], ref[~touched], tol[~touched], "prefill")
    dec = _handle(ds4, "bf16", heads, kv, dim, window, sink, 1, 2)
    for length in (300, 200, 151, 152, 100):
        qd = torch.randn(1, 2, heads, dim, generator=g).bfloat16().cuda()
        o = dec.decode(cache, qd, torch.tensor([length], dtype=torch.int32).cuda())
        ref, tol = attention(qd[0], gather(kc, table, 0, length), gather(vc, table, 0, length), length - 2, window, sink,
                             dim ** -0.5)
        for j in range(2):
            i = length - 2 + j
            if not any(pos <= i and pos > i - window for pos in (100, 101, 250)):
                _check(o[0, j], ref[j], tol[j], f"decode at {i}")


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (64, 1, 512), (64, 2, 64)])
def test_seen_nan_and_infinity_show(heads, kv, dim):
    """What a row sees reaches it: a NaN key or value gives NaN, an infinite
    value gives infinity in its element."""
    ds4 = _ds4()
    n = 200
    for where, bad in (("k", math.nan), ("v", math.nan), ("v", math.inf)):
        k, v, table = paged([n], 16, kv, dim, torch.bfloat16, 12)
        (k if where == "k" else v)[table[0, 5], 3, :, 2] = bad
        kd, vd = to_cuda(k, v)
        q = torch.randn(1, 1, heads, dim, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        at = _handle(ds4, "bf16", heads, kv, dim, 0, 0, 1, 1)
        out = at.decode(ds4.KVCache(kd, vd, table.cuda()), q, torch.tensor([n], dtype=torch.int32).cuda())
        if where == "k":
            assert torch.isnan(out).all()
        elif bad == math.inf:
            assert torch.isinf(out[..., 2]).all() and torch.isfinite(out[..., 3:]).all()
        else:
            assert torch.isnan(out[..., 2]).all() and torch.isfinite(out[..., 3:]).all()


def test_keys_and_values_in_the_same_memory():
    ds4 = _ds4()
    k, _, table = paged([333], 64, 1, 512, torch.bfloat16, 2)
    kd = k.cuda()
    q = torch.randn(1, 2, 64, 512).bfloat16().cuda()
    at = _handle(ds4, "bf16", 64, 1, 512, 0, 0, 1, 2)
    out = at.decode(ds4.KVCache(kd, kd, table.cuda()), q, torch.tensor([333], dtype=torch.int32).cuda())
    kk = gather(kd, table, 0, 333)
    ref, tol = attention(q[0], kk, kk, 331, 0, 0, 512 ** -0.5)
    _check(out[0], ref, tol)


def test_offsets_past_32_bits():
    """Pages at the end of pools of more than 2^32 elements (9 GB each)."""
    ds4 = _ds4()
    for heads, kv, dim in [(8, 2, 128), (64, 1, 512)]:
        page, n = 128, 300
        n_pages = 2 ** 32 // (page * kv * dim) + 8
        kd = torch.zeros(n_pages, page, kv, dim, dtype=torch.bfloat16, device="cuda")
        vd = torch.zeros_like(kd)
        table = torch.tensor([[n_pages - 1, n_pages - 7, n_pages - 3]], dtype=torch.int32)
        at = _handle(ds4, "bf16", heads, kv, dim, 0, 0, 1, n)
        cache = ds4.KVCache(kd, vd, table.cuda())
        kn, vn = torch.randn(n, kv, dim).cuda(), torch.randn(n, kv, dim).cuda()
        length = torch.tensor([n], dtype=torch.int32).cuda()
        at.append(cache, kn, vn, length)
        q = torch.randn(1, 1, heads, dim).bfloat16().cuda()
        out = at.decode(cache, q, length)
        assert at.device_error() == 0
        ref, tol = attention(q[0], kn.bfloat16(), vn.bfloat16(), n - 1, 0, 0, dim ** -0.5)
        _check(out[0], ref, tol)
        qp = torch.randn(n, heads, dim).bfloat16().cuda()
        out = at.prefill(cache, qp, torch.tensor([0, n], dtype=torch.int32).cuda(), length)
        ref, tol = attention(qp, kn.bfloat16(), vn.bfloat16(), 0, 0, 0, dim ** -0.5)
        _check(out, ref, tol)
        del kd, vd, cache
        torch.cuda.empty_cache()


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (64, 1, 512), (64, 2, 64)])
def test_bad_pages_and_lengths_raise_flags(heads, kv, dim):
    """Data errors set a flag and leave the handle usable; keys and values of
    a page outside the cache are read as zeros."""
    ds4 = _ds4()
    n = 100
    k, v, table = paged([n], 16, kv, dim, torch.bfloat16, 6)
    kd, vd = to_cuda(k, v)
    q = torch.randn(1, 1, heads, dim).bfloat16().cuda()
    length = torch.tensor([n], dtype=torch.int32).cuda()
    at = _handle(ds4, "bf16", heads, kv, dim, 0, 0, 2, 64)
    good = at.decode(ds4.KVCache(kd, vd, table.cuda()), q, length)
    assert at.device_error() == 0
    kk, vv = gather(kd, table, 0, n).clone(), gather(vd, table, 0, n).clone()
    kk[32:48] = 0
    vv[32:48] = 0
    ref, tol = attention(q[0], kk, vv, n - 1, 0, 0, dim ** -0.5)
    for entry in (-1, -2 ** 31, kd.shape[0], 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 2] = entry
        cache = ds4.KVCache(kd, vd, bad.cuda())
        out = at.decode(cache, q, length)
        assert at.device_error() == ds4.DEVERR_PAGE and at.device_error() == 0
        _check(out[0], ref, tol)
        out = at.prefill(cache, q[0], torch.tensor([0, 1], dtype=torch.int32).cuda(), length)
        assert at.device_error() == ds4.DEVERR_PAGE
        _check(out, ref, tol)
    cache = ds4.KVCache(kd, vd, table.cuda())
    for wrong in (-5, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        at.decode(cache, q, torch.tensor([wrong], dtype=torch.int32).cuda())
        assert at.device_error() & ds4.DEVERR_LENGTH
    for cu in ([0, 99999, 3], [-7, 1, 2], [2, 1, 0]):
        at.prefill(cache_of(ds4, kd, vd, table), q[0].expand(2, -1, -1).contiguous(),
                   torch.tensor(cu, dtype=torch.int32).cuda(), torch.tensor([n, n], dtype=torch.int32).cuda())
        assert at.device_error() & ds4.DEVERR_LENGTH
    assert torch.equal(at.decode(cache, q, length), good)
    assert at.device_error() == 0


def cache_of(ds4, kd, vd, table):
    return ds4.KVCache(kd, vd, torch.cat([table, table]).contiguous().cuda())


def test_table_entries_of_unseen_pages_are_not_read():
    """A window cache that has given its old pages back."""
    ds4 = _ds4()
    for heads, kv, dim in [(8, 2, 128), (64, 1, 512)]:
        n, window, sink = 1000, 130, 20
        k, v, table = paged([n], 16, kv, dim, torch.bfloat16, 6)
        kd, vd = to_cuda(k, v)
        freed = table.clone()
        freed[0, 2:(n - 2 - window + 1) // 16] = -1
        q = torch.randn(1, 2, heads, dim).bfloat16().cuda()
        at = _handle(ds4, "bf16", heads, kv, dim, window, sink, 1, 2)
        out = at.decode(ds4.KVCache(kd, vd, freed.cuda()), q, torch.tensor([n], dtype=torch.int32).cuda())
        assert at.device_error() == 0
        ref, tol = attention(q[0], gather(kd, table, 0, n), gather(vd, table, 0, n), n - 2, window, sink, dim ** -0.5)
        _check(out[0], ref, tol)


def test_streams_and_graphs():
    """A call on a side stream, and a captured step replayed on new data."""
    ds4 = _ds4()
    heads, kv, dim, n = 32, 8, 128, 700
    k, v, table = paged([n], 64, kv, dim, torch.bfloat16, 8)
    kd, vd = to_cuda(k, v)
    cache = ds4.KVCache(kd, vd, table.cuda())
    at = _handle(ds4, "bf16", heads, kv, dim, 0, 0, 1, 64)
    q = torch.randn(1, 1, heads, dim).bfloat16().cuda()
    kn, vn = torch.randn(1, 1, kv, dim).cuda(), torch.randn(1, 1, kv, dim).cuda()
    length = torch.tensor([n], dtype=torch.int32).cuda()
    out, ragged = torch.empty_like(q), torch.empty_like(q[0])
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ref = at.decode(cache, q, length)
    torch.cuda.synchronize()  # one handle, one stream at a time
    other = at.decode(cache, q, length, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(ref, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        at.append(cache, kn, vn, length)
        at.decode(cache, q, length, out=out)
        at.prefill(cache, q[0], cu, length, out=ragged)
    for i in range(3):
        kn.normal_()
        vn.normal_()
        q.normal_()
        length.fill_(n - 100 * i)
        graph.replay()
        torch.cuda.synchronize()
        m = n - 100 * i
        kk, vv = gather(kd, table, 0, m), gather(vd, table, 0, m)
        assert torch.equal(kk[m - 1], kn[0, 0].bfloat16()) and torch.equal(vv[m - 1], vn[0, 0].bfloat16())
        ref, tol = attention(q[0], kk, vv, m - 1, 0, 0, dim ** -0.5)
        _check(out[0], ref, tol, f"replay {i}")
        _check(ragged, ref, tol, f"replay {i}, ragged")
    assert at.device_error() == 0


def test_two_handles_on_two_streams():
    """Handles are independent: their calls may overlap."""
    ds4 = _ds4()
    heads, kv, dim, n = 64, 1, 512, 3000
    k, v, table = paged([n], 64, kv, dim, torch.bfloat16, 8)
    kd, vd = to_cuda(k, v)
    cache = ds4.KVCache(kd, vd, table.cuda())
    q = torch.randn(2, 1, 2, heads, dim).bfloat16().cuda()
    length = torch.tensor([n], dtype=torch.int32).cuda()
    ats = [_handle(ds4, "bf16", heads, kv, dim, 0, 0, 1, 2) for _ in range(2)]
    alone = [ats[0].decode(cache, q[i], length) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for i in range(2):
            outs[i].append(ats[i].decode(cache, q[i], length, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])
        assert ats[i].device_error() == 0


@pytest.mark.parametrize("kind,source", [("bf16", "fp32"), ("bf16", "own"), ("fp16", "fp32"), ("fp16", "own")])
@pytest.mark.parametrize("kv,dim,page", [(1, 512, 128), (8, 128, 16), (3, 64, 48)])
def test_append(kind, source, kv, dim, page):
    """Every new row lands rounded in its place; nothing else changes."""
    ds4 = _ds4()
    dt = DTYPES[kind]
    src = torch.float32 if source == "fp32" else dt
    for runs, ragged in (([(0, 0), (5, 0), (1, 77), (0, 9), (130, 20)], True), ([(3, 0), (3, 100), (3, 15)], False)):
        lens = [n + h for n, h in runs]
        T = sum(n for n, _ in runs)
        k, v, table = paged(lens, page, kv, dim, dt, 5, fill=0.25)
        kd, vd = to_cuda(k, v)
        g = torch.Generator().manual_seed(9)
        kn, vn = torch.randn(T, kv, dim, generator=g).to(src), torch.randn(T, kv, dim, generator=g).to(src)
        kn.view(-1)[:4] = torch.tensor([math.inf, -math.inf, 0.0, -0.0]).to(src)
        at = _handle(ds4, kind, kv, kv, dim, 0, 0, len(runs), T)
        cu = [0]
        for n, _ in runs:
            cu.append(cu[-1] + n)
        at.append(ds4.KVCache(kd, vd, table.cuda()), kn.cuda(), vn.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                  cu_q=torch.tensor(cu, dtype=torch.int32).cuda() if ragged else None)
        assert at.device_error() == 0
        for b, (n, h) in enumerate(runs):
            for j in range(n):
                pos = h + j
                k[table[b, pos // page], pos % page] = kn[cu[b] + j].to(dt)
                v[table[b, pos // page], pos % page] = vn[cu[b] + j].to(dt)
        assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16))
        assert torch.equal(vd.cpu().view(torch.int16), v.view(torch.int16))


def test_append_drops_what_has_no_place():
    ds4 = _ds4()
    k, v, table = paged([40], 16, 2, 64, torch.bfloat16, 5, fill=0.5)
    kd, vd = to_cuda(k, v)
    at = _handle(ds4, "bf16", 2, 2, 64, 0, 0, 1, 8)
    kn = torch.randn(1, 8, 2, 64).cuda()
    for entry, length, flag in ((-1, 40, "PAGE"), (kd.shape[0], 40, "PAGE"), (0, 4, "LENGTH"),
                                (0, table.shape[1] * 16 + 4, "LENGTH")):
        bad = table.clone()
        bad[0, :] = entry
        if flag == "LENGTH":  # the rows with a place are written, the others dropped
            bad[0, :] = 1
        at.append(ds4.KVCache(kd, vd, bad.cuda()), kn, kn, torch.tensor([length], dtype=torch.int32).cuda())
        assert at.device_error() == getattr(ds4, "DEVERR_" + flag)
    untouched = torch.tensor([p for p in range(kd.shape[0]) if p != 1])
    assert torch.equal(kd.cpu()[untouched], k[untouched])


def test_append_keys_only_and_strides():
    ds4 = _ds4()
    k, v, table = paged([20], 16, 2, 64, torch.bfloat16, 5, fill=0.0, layout="heads")
    kd, vd = to_cuda(k, v)
    at = _handle(ds4, "bf16", 2, 2, 64, 0, 0, 1, 20)
    wide = torch.randn(20, 6, 64).cuda()
    at.append(ds4.KVCache(kd, vd, table.cuda()), wide[:, 2:4], None, torch.tensor([20], dtype=torch.int32).cuda())
    assert torch.equal(gather(kd, table, 0, 20), wide[:, 2:4].bfloat16())
    assert torch.equal(vd.cpu(), v)


def test_refusals():
    ds4 = _ds4()
    k, v, table = paged([40], 16, 2, 64, torch.bfloat16, 5)
    kd, vd = to_cuda(k, v)
    cache = ds4.KVCache(kd, vd, table.cuda())
    at = _handle(ds4, "bf16", 4, 2, 64, 0, 0, 1, 17)
    length = torch.tensor([40], dtype=torch.int32).cuda()
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ds4.Ds4MoeError):  # more sequences than the handle's
        at.decode(ds4.KVCache(kd, vd, table.repeat(2, 1).cuda()), q.repeat(2, 1, 1, 1), length.repeat(2))
    with pytest.raises(ds4.Ds4MoeError):  # more new tokens than a decode call takes
        at.decode(cache, q.repeat(1, 17, 1, 1), length)
    with pytest.raises(ds4.Ds4MoeError):  # more rows than the handle's
        at.prefill(cache, q[0].repeat(18, 1, 1), torch.tensor([0, 18], dtype=torch.int32).cuda(), length)
    with pytest.raises(ds4.Ds4MoeError):  # a page size that is not a multiple of 16
        at.decode(ds4.KVCache(kd[:, :8], vd[:, :8], table.cuda()), q, length)
    with pytest.raises(ds4.Ds4MoeError):  # a pool that is not 16-byte aligned
        flat = torch.zeros(kd.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:1 + kd.numel()].view(kd.shape)
        at.decode(ds4.KVCache(flat, vd, table.cuda()), q, length)
    with pytest.raises(ValueError):
        at.decode(cache, q.half(), length)
    with pytest.raises(ValueError):
        at.decode(cache, q[..., :32], length)
    with pytest.raises(ValueError):
        at.decode(cache, q, length.long())
    with pytest.raises(ValueError):
        at.decode(cache, q.cpu(), length)
    with pytest.raises(ValueError):
        at.decode(cache, q, length, out=torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        at.append(cache, torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda"), None, length)
    with pytest.raises(ValueError):
        ds4.KVCache(kd, vd, table.cuda().long())
    with pytest.raises(ValueError):
        ds4.KVCache(kd, vd[:2], table.cuda())
    # empty calls do nothing
    at.prefill(cache, q[0][:0], torch.tensor([0, 0], dtype=torch.int32).cuda(), length)
    assert at.device_error() == 0
