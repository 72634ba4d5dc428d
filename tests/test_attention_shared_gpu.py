"""Decode attention of batches with shared positions (ds4moe_attn_decode_shared)
against the formula in 64 bits, every sequence over its own table."""
import ctypes
import math

import pytest
import torch

from tests.attn_ref import DTYPES, attention, gather

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


def _batch(kind, kv, dim, page, groups, lens, seed, fill=math.nan):
    """groups: (first sequence, end, shared positions). Sequences of a group have
    the whole shared pages in common and a copy each of the page in which the
    shared positions end. Rows past a length hold `fill`."""
    dt = DTYPES[kind]
    g = torch.Generator().manual_seed(seed)
    width = max([-(-n // page) for n in lens] + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    used = {}
    for a, e, s in groups:
        if a >= e:
            continue
        deep = max(lens[a:e])
        common = [torch.randn(min(s, deep), kv, dim, generator=g).to(dt) for _ in range(2)]
        whole = [None] * (s // page)
        for b in range(a, e):
            rows = [torch.cat([c[:lens[b]], torch.randn(max(0, lens[b] - c.shape[0]), kv, dim, generator=g).to(dt)]) for c in common]
            for p in range(-(-lens[b] // page)):
                mine = len(used)
                if p < s // page and lens[b] >= (p + 1) * page:
                    if whole[p] is not None:
                        table[b, p] = whole[p]
                        continue
                    whole[p] = mine
                table[b, p] = mine
                used[mine] = [r[p * page:(p + 1) * page] for r in rows]
    order = torch.randperm(len(used) + 2, generator=g)
    pools = [torch.full((len(order), page, kv, dim), fill, dtype=dt) for _ in range(2)]
    for i, rows in used.items():
        for pool, r in zip(pools, rows):
            pool[order[i], :r.shape[0]] = r
    table = torch.where(table >= 0, order[table.clamp(min=0).long()].int(), table)
    return pools[0].cuda(), pools[1].cuda(), table


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _check(out, q, k, v, table, lens, new, what=""):
    for b, n in enumerate(lens):
        ref, tol = attention(q[b], gather(k, table, b, n), gather(v, table, b, n), n - new, 0, 0, q.shape[-1] ** -0.5)
        got = out[b].double()
        over = (got - ref).abs() - tol
        assert (over <= 0).all(), f"{what} sequence {b} of {n}: {int((~(over <= 0)).sum())} of {over.numel()} off, worst by " \
                                  f"{float(over.max())} (error {float((got - ref).abs().max())})"


def _run(kind, heads, kv, dim, page, groups, lens, new, seed=0, bounds=True, share=True):
    ds4 = _ds4()
    k, v, table = _batch(kind, kv, dim, page, groups, lens, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), new, heads, dim, generator=g) * 1.5).to(DTYPES[kind]).cuda()
    n_tok = len(lens) * new
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, max_seqs=len(lens), max_tokens=n_tok, max_shared_tokens=n_tok))
    at.debug_share(share)
    cache, kv_len = ds4.KVCache(k, v, table.cuda()), _ints(lens)
    shared = _ints([s for _, _, s in groups])
    start = _ints([a for a, _, _ in groups] + [groups[-1][1]]) if bounds else None
    out = at.decode(cache, q, kv_len, shared_len=shared, group_start=start)
    assert at.device_error() == 0
    _check(out, q, k, v, table, lens, new)
    again = at.decode(cache, q, kv_len, shared_len=shared, group_start=start)
    assert torch.equal(out, again), "two calls differ"
    at.close()


SHAPES = [(8, 8, 64, 1), (32, 8, 128, 1), (8, 2, 128, 4), (6, 2, 64, 3), (40, 2, 64, 1), (16, 1, 128, 2), (8, 2, 256, 1),
          (12, 4, 256, 5), (64, 1, 512, 1), (64, 1, 512, 4), (5, 5, 512, 2), (128, 1, 64, 1), (64, 1, 512, 3)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,dim,new", SHAPES)
def test_one_group(kind, heads, kv, dim, new):
    """Own parts from none to some hundred positions, a sequence that ends before
    the shared positions do, an empty one, among them."""
    for s, page in ((300, 16), (512, 64), (128, 32)):
        lens = [s + x for x in (new, new + 1, 17, 128, 129, 500, new - 1)] + [s - 1, 40, 0, s + 64]
        _run(kind, heads, kv, dim, page, [(0, len(lens), s)], lens, new, seed=s + new, bounds=False)


@pytest.mark.parametrize("heads,kv,dim,new", SHAPES)
def test_groups(heads, kv, dim, new):
    """Groups of several sizes, one of a single sequence, one that shares
    nothing, one that shares little, an empty group."""
    groups = [(0, 5, 700), (5, 6, 400), (6, 9, 0), (9, 9, 50), (9, 12, 100), (12, 19, 131)]
    lens = [s + 1 + (37 * b) % 90 + new for a, e, s in groups for b in range(a, e)]
    _run("bf16", heads, kv, dim, 16, groups, lens, new, seed=dim)


@pytest.mark.parametrize("heads,kv,dim,new", [(32, 8, 128, 1), (8, 8, 64, 2), (8, 2, 256, 1), (64, 1, 512, 4), (64, 1, 512, 1)])
def test_long(heads, kv, dim, new):
    """Shared positions split over many blocks, own parts longer than them."""
    _run("bf16", heads, kv, dim, 64, [(0, 6, 20011)], [20011 + x for x in (5, 3000, 17, new, 700, 64)], new, seed=3)
    _run("fp16", heads, kv, dim, 128, [(0, 3, 513), (3, 5, 4000)], [9000, 513 + new, 12345, 4100, 8000], new, seed=4)


@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 128), (8, 1, 256), (64, 1, 512), (16, 4, 64)])
def test_many_sequences(heads, kv, dim):
    """More sequences, groups and row groups than a block walks through itself."""
    groups = [(3 * i, 3 * i + 3, 128 + (i * 29) % 200) for i in range(45)]
    lens = [s + 1 + (11 * b) % 60 for a, e, s in groups for b in range(a, e)]
    _run("bf16", heads, kv, dim, 16, groups, lens, 1, seed=5)
    lens = [260 + (7 * b) % 40 for b in range(700)]
    _run("bf16", heads, kv, dim, 16, [(0, 700, 250)], lens, 1, seed=6, bounds=False)


@pytest.mark.parametrize("heads,kv,dim,new", [(32, 8, 128, 1), (16, 4, 64, 2), (64, 8, 128, 4), (8, 2, 256, 1), (64, 1, 512, 1), (64, 1, 512, 4)])
def test_where_it_gains(heads, kv, dim, new):
    """Without the test hook: groups that share and groups that do not in one
    batch, and a batch that gains nothing, which is the plain call."""
    _run("bf16", heads, kv, dim, 64, [(0, 12, 9000), (12, 14, 300), (14, 15, 3000), (15, 30, 8000)],
         [s + 10 + (37 * b) % 200 for a, e, s in ((0, 12, 9000), (12, 14, 300), (14, 15, 3000), (15, 30, 8000)) for b in range(a, e)],
         new, seed=15, share=False)
    ds4, at, cache, k, v, table, q, lens = _setup(heads, kv, dim, new, own=(5, 30, 64, max(2, new)))
    at.debug_share(False)
    counts = [at.launch_count()]
    plain = at.decode(cache, q, _ints(lens))
    counts.append(at.launch_count())
    assert torch.equal(plain, at.decode(cache, q, _ints(lens), shared_len=_ints([200])))
    assert at.launch_count() - counts[1] == counts[1] - counts[0]


def test_pages():
    for page in (16, 48, 256, 1024):
        for heads, kv, dim, new in ((8, 2, 128, 1), (64, 1, 512, 1), (32, 2, 64, 4)):
            _run("bf16", heads, kv, dim, page, [(0, 4, 3 * page // 2 + 130)], [3 * page // 2 + 130 + x for x in (4, page, 50, 2 * page + 1)],
                 new, seed=page)


def _setup(heads=8, kv=2, dim=128, new=2, s=200, own=(5, 30, 64, 2), page=16, kind="bf16", seed=9, fill=math.nan, **kw):
    ds4 = _ds4()
    lens = [s + x for x in own]
    k, v, table = _batch(kind, kv, dim, page, [(0, len(lens), s)], lens, seed, fill)
    q = (torch.randn(len(lens), new, heads, dim, generator=torch.Generator().manual_seed(seed)) * 1.5).to(DTYPES[kind]).cuda()
    n = len(lens) * new
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, max_seqs=len(lens), max_tokens=n + 4, max_shared_tokens=n, **kw))
    at.debug_share()
    return ds4, at, ds4.KVCache(k, v, table.cuda()), k, v, table, q, lens


SMALL = [(8, 2, 128, 2), (6, 2, 64, 3), (8, 1, 256, 2), (64, 1, 512, 4), (64, 1, 512, 1)]


@pytest.mark.parametrize("heads,kv,dim,new", SMALL)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite(heads, kv, dim, new, bad):
    """At a shared position every row has it; at an own position the rows from
    there on, and no other row; past a length no row."""
    ds4, at, cache, k, v, table, q, lens = _setup(heads, kv, dim, new, own=(5, 30, 64, max(2, new)))
    n = _ints(lens)
    clean = at.decode(cache, q, n, shared_len=_ints([200]))
    # the last position of sequence 1: only its last new token sees it
    p = lens[1] - 1
    page, row = int(table[1, p // 16]), p % 16
    keep = v[page, row].clone()
    v[page, row] = bad
    out = at.decode(cache, q, n, shared_len=_ints([200]))
    assert (~torch.isfinite(out[1, -1].float())).all()
    assert torch.isfinite(out[1, :-1].float()).all()
    if new > 1:
        _check(out[1:2, :-1], q[1:2, :-1], k, v, table[1:2], [lens[1] - 1], new - 1)
    for b in (0, 2, 3):
        assert torch.equal(out[b], clean[b])
    v[page, row] = keep
    page = int(table[0, 2])
    v[page, 3, 0, 5] = bad
    out = at.decode(cache, q, n, shared_len=_ints([200]))
    g = heads // kv
    assert (~torch.isfinite(out[:, :, :g, 5].float())).all()
    rest = out.clone()
    rest[:, :, :g, 5] = clean[:, :, :g, 5]
    assert torch.equal(rest, clean)
    assert at.device_error() == 0


@pytest.mark.parametrize("heads,kv,dim,new", SMALL)
def test_scores_of_minus_infinity(heads, kv, dim, new):
    """All shared scores -infinity: the own positions' result; all own ones: the
    shared positions'; all: zeros."""
    ds4, at, cache, k, v, table, q, lens = _setup(heads, kv, dim, new, s=208, own=(5, 30, 64, max(2, new)), page=16)
    q.abs_()
    kk = k.clone()
    shared_pages = table[0, :13].long().cuda()
    own_pages = torch.tensor([int(x) for row in table[:, 13:] for x in row if x >= 0]).cuda()

    def masked(pages):
        k.copy_(kk)
        for p in pages:
            k[p] = torch.where(torch.isnan(k[p]), k[p], -math.inf)
        return at.decode(cache, q, _ints(lens), shared_len=_ints([208]))
    only_own = masked(shared_pages)
    _check(only_own, q, kk, v, table[:, 13:], [n - 208 for n in lens], new, "own")
    only_shared = masked(own_pages)
    for b in range(len(lens)):
        # every row sees all shared positions: as new rows of a sequence that ends with them
        for j in range(new):
            ref, tol = attention(q[b, j:j + 1], gather(kk, table, b, 208), gather(v, table, b, 208), 207, 0, 0, dim ** -0.5)
            assert ((only_shared[b, j:j + 1].double() - ref).abs() <= tol).all()
    none = masked(torch.cat([shared_pages, own_pages]))
    assert (none == 0).all()
    assert at.device_error() == 0


def test_a_nan_that_long_rows_do_not_see():
    """Rows of more than 65536 positions are computed once more in a launch of
    their own."""
    for heads, kv, dim, new in ((8, 1, 256, 2), (40, 2, 64, 2)):
        ds4 = _ds4()
        s, lens = 66000, [66010, 66100]
        k, v, table = _batch("bf16", kv, dim, 1024, [(0, 2, s)], lens, 21)
        q = (torch.randn(2, new, heads, dim, generator=torch.Generator().manual_seed(2)) * 1.5).bfloat16().cuda()
        at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, max_seqs=2, max_tokens=4, max_shared_tokens=4))
        at.debug_share()
        p = lens[0] - 1
        v[int(table[0, p // 1024]), p % 1024] = math.nan
        out = at.decode(ds4.KVCache(k, v, table.cuda()), q, _ints(lens), shared_len=_ints([s]))
        assert torch.isnan(out[0, -1]).all()
        _check(out[:1, :-1], q[:1, :-1], k, v, table[:1], [lens[0] - 1], new - 1, "before the NaN")
        _check(out[1:], q[1:], k, v, table[1:], lens[1:], new, "beside it")
        assert at.device_error() == 0


def test_lengths_bounds_and_pages_out_of_range():
    ds4, at, cache, k, v, table, q, lens = _setup(own=(5, 30, 64, 2, 9, 40))
    assert ds4.lib().ds4moe_attn_debug_share(None, 1) == 1 and ds4.lib().ds4moe_attn_debug_share(at._h, 2) == 1
    # bounds out of order: each is raised to the largest before it, sequences never belong to two groups
    out = at.decode(cache, q, _ints(lens), shared_len=_ints([200, 190, 150]), group_start=_ints([0, 4, 2, 6]))
    _check(out, q, k, v, table, lens, 2)
    assert at.device_error() == ds4.DEVERR_LENGTH
    out = at.decode(cache, q, _ints(lens), shared_len=_ints([200, 200]), group_start=_ints([-3, 3, 99]))
    _check(out, q, k, v, table, lens, 2)
    assert at.device_error() == ds4.DEVERR_LENGTH
    # bounds that leave sequences out are fine
    out = at.decode(cache, q, _ints(lens), shared_len=_ints([200]), group_start=_ints([2, 5]))
    _check(out, q, k, v, table, lens, 2)
    assert at.device_error() == 0
    for s, flag in ((-5, ds4.DEVERR_LENGTH), (10 ** 9, ds4.DEVERR_LENGTH), (0, 0)):
        out = at.decode(cache, q, _ints(lens), shared_len=_ints([s]))
        _check(out, q, k, v, table, lens, 2)
        assert at.device_error() == flag
    # a bad page under the shared positions reads as zeros
    bad = table.clone()
    bad[:, 3] = 10 ** 6
    out = at.decode(ds4.KVCache(k, v, bad.cuda()), q, _ints(lens), shared_len=_ints([200]))
    assert at.device_error() == ds4.DEVERR_PAGE
    kz, vz = k.clone(), v.clone()
    kz[int(table[0, 3])] = 0
    vz[int(table[0, 3])] = 0
    _check(out, q, kz, vz, table, lens, 2)


def test_an_empty_place_before_the_others():
    """The first sequence of the batch is empty and has no table: the next one's
    is read."""
    ds4, at, cache, k, v, table, q, lens = _setup(own=(5, 30, 64, 2))
    gone = table.clone()
    gone[0] = -1
    n = [0] + lens[1:]
    out = at.decode(ds4.KVCache(k, v, gone.cuda()), q, _ints(n), shared_len=_ints([200]))
    assert at.device_error() == 0 and (out[0] == 0).all()
    _check(out[1:], q[1:], k, v, table[1:], lens[1:], 2)
    out = at.decode(ds4.KVCache(k, v, gone.cuda()), q, _ints([1] + lens[1:]), shared_len=_ints([200]), group_start=_ints([1, 4]))
    assert at.device_error() == ds4.DEVERR_PAGE
    _check(out[1:], q[1:], k, v, table[1:], lens[1:], 2)


def test_with_a_window_it_is_the_plain_call():
    for sink in (0, 4):
        ds4, at, cache, k, v, table, q, lens = _setup(window=40, n_sink=sink)
        assert torch.equal(at.decode(cache, q, _ints(lens), shared_len=_ints([200])), at.decode(cache, q, _ints(lens)))


@pytest.mark.parametrize("heads,kv,dim,new", SMALL)
def test_captured_and_on_another_stream(heads, kv, dim, new):
    ds4, at, cache, k, v, table, q, lens = _setup(heads, kv, dim, new, own=(5, 30, 64, max(2, new)))
    n, shared = _ints(lens), _ints([200])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = at.decode(cache, q, n, stream=side, shared_len=shared)
    torch.cuda.current_stream().wait_stream(side)
    _check(out, q, k, v, table, lens, new)
    for bounds in (None, _ints([0, len(lens)])):
        out.zero_()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            at.decode(cache, q, n, out=out, shared_len=shared, group_start=bounds)
        for s, cut in ((200, 0), (136, 3), (0, 1), (199, 0)):  # read when the graph runs
            shared.fill_(s)
            now = [max(x - cut, 0) for x in lens]
            n.copy_(_ints(now))
            g.replay()
            torch.cuda.synchronize()
            _check(out, q, k, v, table, now, new, f"{s} shared")
        n.copy_(_ints(lens)), shared.fill_(200)


def test_strided_rows():
    """q and out within wider rows; what lies between them stays."""
    for heads, kv, dim, new in SMALL:
        ds4, at, cache, k, v, table, q, lens = _setup(heads, kv, dim, new, own=(5, 30, 64, max(2, new)))
        wide = torch.full((len(lens), new, heads + 2, dim), 3.0, dtype=q.dtype).cuda()
        qw = torch.full_like(wide, 2.0)
        qw[:, :, 1:-1] = q
        out = at.decode(cache, qw[:, :, 1:-1], _ints(lens), out=wide[:, :, 1:-1], shared_len=_ints([200]))
        _check(out, q, k, v, table, lens, new)
        assert (wide[:, :, 0] == 3).all() and (wide[:, :, -1] == 3).all()


def test_refusals():
    ds4, at, cache, k, v, table, q, lens = _setup()
    n, s = _ints(lens), _ints([200])
    for kw in (dict(group_start=_ints([0, 4])), dict(shared_len=s.long()), dict(shared_len=s.cpu()), dict(shared_len=s, group_start=_ints([0])),
               dict(shared_len=s, group_start=_ints([0, 2, 4]))):
        with pytest.raises(ValueError):
            at.decode(cache, q, n, **kw)
    with pytest.raises(ds4.Ds4MoeError):
        at.decode(cache, q, n, shared_len=_ints([200, 200]))  # two groups without bounds
    with pytest.raises(ds4.Ds4MoeError):
        at.decode(cache, q, n, shared_len=_ints([1] * 5), group_start=_ints([0, 1, 2, 3, 4, 4]))  # more groups than sequences
    with pytest.raises(ds4.Ds4MoeError):
        at.decode(cache, q, n, shared_len=s[:0])
    bare = ds4.Attention(ds4.AttentionDesc(8, 2, 128, max_seqs=4, max_tokens=8))
    with pytest.raises(ds4.Ds4MoeError):
        bare.decode(cache, q, n, shared_len=s)  # nothing reserved
    with pytest.raises(ds4.Ds4MoeError):
        ds4.Attention(ds4.AttentionDesc(8, 2, 128, max_seqs=4, max_tokens=8, max_shared_tokens=9))
    L = ds4.lib()
    assert L.ds4moe_attn_reserve_shared(None, 1) == 1 and L.ds4moe_attn_reserve_shared(bare._h, -1) == 1
    before = bare.device_bytes()
    assert L.ds4moe_attn_reserve_shared(bare._h, 4) == 0 and bare.device_bytes() > before
    with pytest.raises(ds4.Ds4MoeError):
        bare.decode(cache, q, n, shared_len=s)  # more rows than reserved
    assert L.ds4moe_attn_reserve_shared(bare._h, 8) == 0 and L.ds4moe_attn_reserve_shared(bare._h, 2) == 0
    bare.debug_share()
    assert torch.equal(bare.decode(cache, q, n, shared_len=s), at.decode(cache, q, n, shared_len=s))
    p = ctypes.c_void_p
    row = 8 * 128
    good = [at._h, cache.ref, p(q.data_ptr()), row, p(n.data_ptr()), p(s.data_ptr()), None, 1, 4, 2, p(torch.empty_like(q).data_ptr()), row, None]
    for i, bad in ((0, None), (1, None), (2, None), (3, 100), (4, None), (5, None), (7, 0), (7, 2), (8, -1), (8, 5), (9, 0), (9, 17), (10, None)):
        assert L.ds4moe_attn_decode_shared(*[bad if j == i else x for j, x in enumerate(good)]) == 1, (i, bad)
