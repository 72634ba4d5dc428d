"""NaN and infinities in keys and values: what a row sees shows in it, what it
does not see never does, and neither makes a call slow or unfinished."""
import math

import pytest
import torch

from tests.attn_ref import attention, gather, paged, to_cuda

pytestmark = pytest.mark.gpu

SHAPES = [(8, 2, 128), (4, 4, 64), (4, 1, 256), (16, 1, 512)]


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


def _setup(n, kv, dim, bad, where, seed=3):
    """A cache of n positions with `bad` = {position: value} in element 5 of
    the values (where "v") or the keys ("k"); clean copies for the formula."""
    k, v, table = paged([n], 32, kv, dim, torch.bfloat16, seed)
    kc, vc = to_cuda(k, v)
    for pos, x in bad.items():
        (v if where == "v" else k)[table[0, pos // 32], pos % 32, :, 5] = x
    kd, vd = to_cuda(k, v)
    return gather(kc, table, 0, n), gather(vc, table, 0, n), kd, vd, table


def _expect(got, q, kc, vc, first, window, sink, bad, where):
    """Rows that see none of `bad` follow the formula; of the others, a key
    makes the row NaN, a value its element 5 only (NaN, or the infinity where
    all that the row sees are the same one)."""
    n, dim = q.shape[0], q.shape[2]
    ref, tol = attention(q, kc, vc, first, window, sink, dim ** -0.5)
    got = got.double()
    ok = (got - ref).abs() <= tol
    for j in range(n):
        i = first + j
        seen = [x for pos, x in bad.items() if pos <= i and (window == 0 or pos > i - window or pos < sink)]
        if not seen:
            assert ok[j].all(), f"position {i}: {int((~ok[j]).sum())} elements off"
        elif where == "k":
            assert torch.isnan(got[j]).all(), f"position {i}"
        else:
            rest = torch.ones(dim, dtype=torch.bool)
            rest[5] = False
            assert ok[j][:, rest].all(), f"position {i}"
            if any(math.isnan(x) for x in seen) or len(set(seen)) > 1:
                assert torch.isnan(got[j][:, 5]).all(), f"position {i}"
            else:
                assert (got[j][:, 5] == seen[0]).all(), f"position {i}"


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("window,sink", [(0, 0), (300, 4), (1500, 40)])
def test_prefill_seen_and_unseen(heads, kv, dim, window, sink, where):
    """Positions at the start, inside a tile and at its end, behind the window
    and among the padding of the first positions; items of one block, and
    items that are joined."""
    ds4 = _ds4()
    T = 2500
    for bad in ({3: math.nan}, {41: math.nan, 1500: math.inf}, {7: math.inf, 1407: math.inf, 1408: -math.inf},
                {T - 1: math.nan}, {j: math.nan for j in range(1111, T)}):
        if where == "k":
            bad = {j: math.nan for j in bad}
        kc, vc, kd, vd, table = _setup(T, kv, dim, bad, where)
        q = torch.randn(T, heads, dim, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, window=window, n_sink=sink, max_tokens=T))
        got = at.prefill(ds4.KVCache(kd, vd, table.cuda()), q, torch.tensor([0, T], dtype=torch.int32).cuda(),
                         torch.tensor([T], dtype=torch.int32).cuda())
        assert at.device_error() == 0
        _expect(got, q, kc, vc, 0, window, sink, bad, where)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("heads,kv,dim,new", [(8, 2, 128, 4), (4, 4, 64, 1), (4, 4, 64, 16), (32, 2, 64, 3), (4, 1, 256, 5),
                                              (64, 1, 512, 4), (64, 1, 512, 1)])
@pytest.mark.parametrize("window,sink", [(0, 0), (300, 4), (1500, 40)])
def test_decode_seen_and_unseen(heads, kv, dim, new, window, sink, where):
    ds4 = _ds4()
    n = 3001
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, window=window, n_sink=sink, max_tokens=new))
    q = torch.randn(1, new, heads, dim, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    for bad in ({3: math.nan}, {41: math.nan, 1500: math.inf}, {n - 1: math.nan}, {n - 2: math.inf, 2900: math.inf},
                {n - 301: math.nan}, {n - 300: -math.inf}, {n - 1501: math.nan, n - 1500: math.inf}):
        if where == "k":
            bad = {j: math.nan for j in bad}
        kc, vc, kd, vd, table = _setup(n, kv, dim, bad, where)
        got = at.decode(ds4.KVCache(kd, vd, table.cuda()), q, torch.tensor([n], dtype=torch.int32).cuda())
        assert at.device_error() == 0
        _expect(got[0], q[0], kc, vc, n - new, window, sink, bad, where)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("heads,kv,dim,T,new", [(32, 8, 128, 2048, 0), (16, 1, 512, 2048, 0), (8, 2, 128, 8192, 2),
                                                (64, 1, 512, 8192, 4)])
def test_seen_nan_is_not_slow(heads, kv, dim, T, new, where):
    """A NaN that every row sees: no row is computed twice. (Computing them
    again takes some hundred times as long; the bound is 10.)"""
    ds4 = _ds4()
    n = new or T
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, max_tokens=n))
    q = torch.randn(n, heads, dim, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    length, cu = torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    times = []
    for bad in ({}, {3: math.nan}):
        kc, vc, kd, vd, table = _setup(T, kv, dim, bad, where)
        cache = ds4.KVCache(kd, vd, table.cuda())

        def call():
            return at.decode(cache, q[None], length)[0] if new else at.prefill(cache, q, cu, length)
        out = call()
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        assert at.device_error() == 0
    seen = out[4:] if not new else out
    assert torch.isnan(seen if where == "k" else seen[..., 5]).all()
    assert times[1] < 10 * times[0], times


@pytest.mark.parametrize("heads,dim,new,members", [(16, 64, 2, 1), (64, 512, 4, 4)])
def test_long_rows_of_unsplit_sequences(heads, dim, new, members):
    """A sequence per block (or per blocks that share its keys), each with a NaN
    value at its last position: rows of 65600 positions, which are computed
    once more after the call's other work."""
    ds4 = _ds4()
    n, page = 65600, 64
    B = torch.cuda.get_device_properties(0).multi_processor_count // members
    per = n // page
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn(2, B * per, page, 1, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    clean = pool[1, per - 1::per, -1, :, 5].clone()
    pool[1, per - 1::per, -1, :, 5] = math.nan
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    q = torch.randn(B, new, heads, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    at = ds4.Attention(ds4.AttentionDesc(heads, 1, dim, max_seqs=B, max_tokens=B * new))
    length = torch.full((B,), n, dtype=torch.int32, device="cuda")
    cache = ds4.KVCache(pool[0], pool[1], table)
    got = at.decode(cache, q, length)
    assert at.device_error() == 0
    assert torch.isfinite(got[:, :-1]).all() and torch.isnan(got[:, -1, :, 5]).all()
    again = at.decode(cache, q, length)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    pool[1, per - 1::per, -1, :, 5] = clean
    for b in (0, 1, B // 2, B - 1):
        ref, tol = attention(q[b], gather(pool[0], table, b, n), gather(pool[1], table, b, n), n - new, 0, 0, dim ** -0.5)
        assert ((got[b].double() - ref).abs() <= tol)[:-1].all(), f"sequence {b}"
        assert ((got[b].double() - ref).abs() <= tol)[-1, :, 6:].all(), f"sequence {b}"
    assert torch.isfinite(at.decode(cache, q, length)).all()  # nothing is left of the earlier call
