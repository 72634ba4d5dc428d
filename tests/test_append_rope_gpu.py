"""The append with the position rotation (ds4moe_kv_append_rope) against its
formula in 64 bits, with angles reduced exactly."""
import math
from fractions import Fraction

import pytest
import torch

from tests.attn_ref import DTYPES, half_step

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)


def _angle(pos, f):
    """pos * f modulo one turn, in radians."""
    if not math.isfinite(f):
        return math.nan
    t = Fraction(pos) * Fraction(f) / (2 * PI)
    return 2 * math.pi * float(t - math.floor(t))


def _rotated(x, pos, freq, offset, interleaved, scale, dt):
    """x [n, heads, dim] (any type) at positions pos, in 64 bits, and the error
    that 32-bit arithmetic and one rounding to dt may make. Cosine and sine: the
    reduced angle is off by pi (2^-26 + 2^-32), the functions by 2 units in the
    last place (2^-23), the scale's product rounds once: below 2^-22 in all. Two
    products and their sum add three roundings of 2^-24."""
    x = x.double().cpu()
    ang = torch.tensor([[_angle(int(p), float(f)) for f in freq] for p in pos], dtype=torch.float64)
    c, s = (torch.cos(ang) * scale)[:, None], (torch.sin(ang) * scale)[:, None]
    half = len(freq)
    i = torch.arange(half)
    ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
    a, b = x[:, :, ia], x[:, :, ib]
    ref, err = x.clone(), torch.zeros_like(x)
    ref[:, :, ia], ref[:, :, ib] = a * c - b * s, b * c + a * s
    err[:, :, ia] = err[:, :, ib] = (a.abs() + b.abs()) * abs(scale) * (2.0 ** -22 + 3 * 2.0 ** -24)
    u = half_step(dt)
    return ref, err * (1 + u) + u * ref.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def _close(got, ref, tol, what):
    got = got.double().cpu()
    same = torch.isnan(got) & torch.isnan(ref)
    over = torch.where(same, -1.0, (got - ref).abs() - tol)
    assert (over <= 0).all(), f"{what}: {int((~(over <= 0)).sum())} of {got.numel()} off"


def _setup(kind, source, heads, kv, dim, page, lens, runs, seed, pages_to_spare=2, scale=1.0, freq=None, rot=None,
           offset=0, interleaved=False, ragged=True, width=None):
    """Sequences of lens[b] positions, the last runs[b] of them new; only the
    pages that are written exist. Cache and q_out hold 7 at first."""
    import deepseek_v4_flash_gb300 as ds4
    dt = DTYPES[kind]
    src = torch.float32 if source == "fp32" else dt
    g = torch.Generator().manual_seed(seed)
    n_tok = sum(runs)
    rot = rot or dim
    if freq is None:
        freq = 1.0 / 10000.0 ** (torch.arange(0, rot, 2, dtype=torch.float32) / rot)
    need = [(b, p) for b in range(len(lens)) for p in range(max(0, lens[b] - runs[b]) // page, -(-lens[b] // page))]
    order = torch.randperm(len(need) + pages_to_spare, generator=g)
    width = width or max([-(-n // page) for n in lens] + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for i, (b, p) in enumerate(need):
        table[b, p] = int(order[i])
    shape = (len(order), page, kv, dim)
    k, v = torch.full(shape, 7.0, dtype=dt), torch.full(shape, 7.0, dtype=dt)
    new = [torch.randn(n_tok, h, dim, generator=g).to(src) for h in (heads, kv, kv)]
    cu = torch.tensor([0] + torch.tensor(runs).cumsum(0).tolist(), dtype=torch.int32)
    kd, vd = k.cuda(), v.cuda()
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, max_seqs=len(lens), max_tokens=max(n_tok, 1) + 8))
    return dict(ds4=ds4, dt=dt, table=table, kd=kd, vd=vd, new=new, freq=freq, cu=cu, at=at, lens=lens, runs=runs,
                page=page, cache=ds4.KVCache(kd, vd, table.cuda()),
                rope=ds4.Rope(freq.cuda(), offset, interleaved, scale), offset=offset, interleaved=interleaved,
                scale=scale, kv_len=torch.tensor(lens, dtype=torch.int32).cuda())


def _expect(t, skip=()):
    """Expected (q, k, v) pools and their tolerances."""
    pos = [p for b in range(len(t["lens"])) for p in range(t["lens"][b] - t["runs"][b], t["lens"][b])]
    args = (pos, t["freq"].tolist(), t["offset"], t["interleaved"], t["scale"], t["dt"])
    q, qt = _rotated(t["new"][0], *args)
    kk, kt = _rotated(t["new"][1], *args)
    k = torch.full(t["kd"].shape, 7.0, dtype=torch.float64)
    v, ktol = k.clone(), torch.zeros_like(k)
    r = 0
    for b, n in enumerate(t["runs"]):
        for p in range(t["lens"][b] - n, t["lens"][b]):
            if p >= 0 and r not in skip:
                page = int(t["table"][b, p // t["page"]])
                k[page, p % t["page"]], ktol[page, p % t["page"]] = kk[r], kt[r]
                v[page, p % t["page"]] = t["new"][2][r].to(t["dt"]).double()
            r += 1
    return q, qt, k, ktol, v


def _check(t, q_out, flags=0, skip=(), values=True):
    q, qt, k, kt, v = _expect(t, skip)
    assert t["at"].device_error() == flags
    if q_out is not None:
        _close(q_out, q, qt, "queries")
    _close(t["kd"], k, kt, "keys")
    if values:
        assert torch.equal(t["vd"].double().cpu(), v), "values"


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("source", ["fp32", "same"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rot,offset", [(8, 2, 64, 64, 0), (4, 4, 128, 32, 0), (6, 1, 128, 48, 40),
                                                     (3, 3, 256, 256, 0), (64, 1, 512, 64, 448), (5, 1, 512, 16, 8)])
def test_ragged(kind, source, interleaved, heads, kv, dim, rot, offset):
    """Runs of every kind: empty, one token, past a page's end."""
    t = _setup(kind, source if source == "fp32" else kind, heads, kv, dim, 16, [37, 0, 1, 200, 16, 5], [20, 0, 1, 33, 16, 0],
               heads + rot, rot=rot, offset=offset, interleaved=interleaved, scale=1.25 if interleaved else 1.0)
    q_out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], cu_q=t["cu"].cuda(),
                           rope=t["rope"], q=t["new"][0].cuda())
    assert q_out.dtype == t["dt"]
    _check(t, q_out)


@pytest.mark.parametrize("n_seq,new,heads,kv,dim", [(1, 1, 64, 1, 512), (64, 1, 32, 8, 128), (7, 5, 6, 2, 64), (300, 3, 32, 8, 128)])
def test_even_rows(n_seq, new, heads, kv, dim):
    """[n_seq, n_new] rows without bounds; the last is large enough for eight rows a thread."""
    lens = [new + (97 * b) % 50 for b in range(n_seq)]
    t = _setup("bf16", "fp32", heads, kv, dim, 64, lens, [new] * n_seq, 3, rot=16 if n_seq == 300 else None)
    q, k, v = (x.cuda().view(n_seq, new, *x.shape[1:]) for x in t["new"])
    q_out = t["at"].append(t["cache"], k, v, t["kv_len"], rope=t["rope"], q=q)
    assert q_out.shape == q.shape
    _check(t, q_out.flatten(0, 1))


def test_far_positions():
    """Up to the last position that a table can hold."""
    page, width = 65536, 32767
    lens = [page * width, page * width - 70000, 1 << 24, 3]
    freq = torch.tensor([1.0, 0.7391, 1e-3, 3.25e-5, 0.0, -0.31, 1.5e-42, 97.3], dtype=torch.float32)
    t = _setup("bf16", "fp32", 2, 1, 64, page, lens, [3, 2, 2, 3], 4, freq=freq, rot=16, offset=8, width=width)
    q_out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], cu_q=t["cu"].cuda(),
                           rope=t["rope"], q=t["new"][0].cuda())
    _check(t, q_out)


def test_frequencies_that_are_not_finite():
    freq = torch.tensor([math.inf, 0.5, math.nan, 0.25, -math.inf, 1.0, 2.0, 3.0], dtype=torch.float32)
    t = _setup("fp16", "fp32", 2, 1, 64, 16, [5], [5], 5, freq=freq, rot=16)
    q_out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], rope=t["rope"], q=t["new"][0].cuda())
    assert torch.isnan(q_out[..., 0]).all() and torch.isfinite(q_out[..., 1]).all()
    _check(t, q_out)


def test_without_queries_or_values_and_in_place():
    t = _setup("bf16", "bf16", 4, 2, 64, 16, [20, 9], [4, 4], 6)
    none = t["at"].append(t["cache"], t["new"][1].cuda().view(2, 4, 2, 64), None, t["kv_len"], rope=t["rope"])
    assert none is None
    _check(t, None, values=False)
    assert (t["vd"] == 7).all()
    t = _setup("bf16", "bf16", 4, 2, 64, 16, [20, 9], [4, 4], 6)
    q = t["new"][0].cuda()
    got = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], rope=t["rope"], q=q, q_out=q)
    assert got is q
    _check(t, q)


def test_strided_rows():
    """q, k and v as slices of one projection's rows; q_out within wider rows."""
    t = _setup("fp16", "fp32", 4, 2, 64, 16, [20, 9, 40], [5, 2, 30], 7, rot=32)
    rows = torch.cat([x.flatten(1) for x in t["new"]], 1).cuda()
    q, k, v = rows[:, :256].unflatten(1, (4, 64)), rows[:, 256:384].unflatten(1, (2, 64)), rows[:, 384:].unflatten(1, (2, 64))
    wide = torch.full((37, 8, 64), 3.0, dtype=torch.float16).cuda()
    got = t["at"].append(t["cache"], k, v, t["kv_len"], cu_q=t["cu"].cuda(), rope=t["rope"], q=q, q_out=wide[:, 2:6])
    _check(t, got)
    assert (wide[:, :2] == 3).all() and (wide[:, 6:] == 3).all()


@pytest.mark.parametrize("lens, runs", [([20, 9, 40], [5, 2, 30]), ([17], [1])])
def test_columns_of_one_matrix_in_place(lens, runs):
    """q, k and v as columns of one 16-bit matrix, q turned where it is."""
    t = _setup("bf16", "bf16", 4, 2, 64, 16, lens, runs, 14, rot=32)
    rows = torch.cat([x.flatten(1) for x in t["new"]], 1).cuda()
    before = rows.clone()
    q, k, v = rows[:, :256].unflatten(1, (4, 64)), rows[:, 256:384].unflatten(1, (2, 64)), rows[:, 384:].unflatten(1, (2, 64))
    got = t["at"].append(t["cache"], k, v, t["kv_len"], cu_q=t["cu"].cuda(), rope=t["rope"], q=q, q_out=q)
    _check(t, got)
    assert torch.equal(rows[:, 256:], before[:, 256:])
    for bad in (rows[:, 128:384], rows[:, 64:320]):  # over the keys; over the queries by part
        with pytest.raises(t["ds4"].Ds4MoeError):
            t["at"].append(t["cache"], k, v, t["kv_len"], cu_q=t["cu"].cuda(), rope=t["rope"], q=q, q_out=bad.unflatten(1, (4, 64)))


def test_frequencies_of_any_size():
    """From the smallest to the largest fp32 numbers: turns of a whole number of
    2^64ths, so that cosine and sine stay on the circle."""
    freq = torch.tensor([1e-45, 1e-38, 1e-10, 1e8, 1e20, 5e26, 1e30, 3e38], dtype=torch.float32)
    t = _setup("fp16", "fp32", 2, 1, 64, 16, [5], [5], 5, freq=freq, rot=16)
    q = t["new"][0].cuda()
    out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], rope=t["rope"], q=q)
    size = (q[..., :8].double() ** 2 + q[..., 8:16].double() ** 2).sqrt()
    got = (out[..., :8].double() ** 2 + out[..., 8:16].double() ** 2).sqrt()
    # two roundings to fp16 of numbers up to size, and 2^-20 of cosine and sine
    assert ((got - size).abs() <= size * (2.0 ** -10.5 + 2.0 ** -20) + 2.0 ** -24).all()
    # the first three turn by 4e-10 at most: numbers up to 8 change by less than 1e-8
    assert ((out - q)[..., :3].abs().double() <= q[..., :3].abs().double() * 2.0 ** -11 + 2.0 ** -25 + 1e-8).all()


def test_rows_of_no_sequence_and_bad_places():
    """Rows behind the last sequence stay as they are; a row that the cache has
    no place for raises a flag and is rotated all the same."""
    t = _setup("bf16", "fp32", 2, 1, 64, 16, [20, 3, 40], [6, 4, 3], 8)
    table = t["table"].clone()
    table[2, 2] = 99  # positions 37 to 39
    cache = t["ds4"].KVCache(t["kd"], t["vd"], table.cuda())
    pad = [torch.cat([x, torch.randn(5, *x.shape[1:])]).cuda() for x in t["new"]]
    q_out = torch.full((18, 2, 64), 5.0, dtype=torch.bfloat16).cuda()
    t["at"].append(cache, pad[1], pad[2], t["kv_len"], cu_q=t["cu"].cuda(), rope=t["rope"], q=pad[0], q_out=q_out)
    ds4 = t["ds4"]
    assert (q_out[13:] == 5).all()
    _check(t, q_out[:13], ds4.DEVERR_PAGE | ds4.DEVERR_LENGTH, skip=(10, 11, 12))


def test_row_bounds_out_of_order():
    """Bounds are raised to the largest before them, as in the plain append."""
    t = _setup("bf16", "fp32", 2, 1, 64, 16, [20, 30, 40], [6, 4, 3], 9)
    cu = torch.tensor([0, 6, 4, 13], dtype=torch.int32).cuda()  # the second is empty, the third from row 6
    q_out = torch.full((13, 2, 64), 5.0, dtype=torch.bfloat16).cuda()
    t["at"].append(t["cache"], t["new"][1].cuda(), None, t["kv_len"], cu_q=cu, rope=t["rope"], q=t["new"][0].cuda(), q_out=q_out)
    pos = list(range(14, 20)) + list(range(33, 40))
    ref, tol = _rotated(t["new"][0], pos, t["freq"].tolist(), 0, False, 1.0, t["dt"])
    _close(q_out, ref, tol, "queries")
    assert t["at"].device_error() & t["ds4"].DEVERR_LENGTH


def test_many_sequences():
    """More than the blocks check themselves."""
    n = 1300
    runs = [b % 3 for b in range(n)]
    lens = [runs[b] + (31 * b) % 40 for b in range(n)]
    t = _setup("bf16", "fp32", 2, 1, 64, 16, lens, runs, 10, rot=16)
    q_out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], cu_q=t["cu"].cuda(),
                           rope=t["rope"], q=t["new"][0].cuda())
    _check(t, q_out)


def test_long_prompt_agrees_with_the_plain_append():
    """Frequencies of 0 turn nothing: the same bits as the append without rotation."""
    t = _setup("bf16", "fp32", 32, 8, 128, 64, [1500, 777], [1500, 777], 11, freq=torch.zeros(64))
    q_out = t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], cu_q=t["cu"].cuda(),
                           rope=t["rope"], q=t["new"][0].cuda())
    k, v = t["kd"].clone(), t["vd"].clone()
    t["kd"].fill_(7.0), t["vd"].fill_(7.0)
    t["at"].append(t["cache"], t["new"][1].cuda(), t["new"][2].cuda(), t["kv_len"], cu_q=t["cu"].cuda())
    assert torch.equal(k, t["kd"]) and torch.equal(v, t["vd"]) and torch.equal(q_out.cpu(), t["new"][0].to(t["dt"]))


def test_captured_and_on_another_stream():
    t = _setup("bf16", "fp32", 4, 2, 64, 16, [20, 9], [3, 3], 12)
    q, k, v = (x.cuda() for x in t["new"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    first = t["at"].append(t["cache"], k, v, t["kv_len"], rope=t["rope"], q=q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _check(t, first)
    q_out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t["at"].append(t["cache"], k, v, t["kv_len"], rope=t["rope"], q=q, q_out=q_out)
    t["kv_len"].add_(2)  # the graph reads the lengths when it runs
    t["lens"] = [22, 11]
    t["kd"].fill_(7.0), t["vd"].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    _check(t, q_out)


def test_refusals():
    import ctypes
    t = _setup("bf16", "fp32", 4, 2, 64, 16, [20, 9], [3, 3], 13)
    ds4, at, cache = t["ds4"], t["at"], t["cache"]
    q, k, v = (x.cuda() for x in t["new"])
    call = lambda rope=t["rope"], **kw: at.append(cache, kw.pop("k", k), kw.pop("v", v), t["kv_len"], rope=rope, **kw)  # noqa: E731
    f = torch.ones(64).cuda()
    for bad in (ds4.Rope(f[:4]), ds4.Rope(f[:12]), ds4.Rope(f[:40]), ds4.Rope(f[:16], offset=40), ds4.Rope(f[:16], offset=4),
                ds4.Rope(f[:16], offset=-8), ds4.Rope(f[:0]), ds4.Rope(f[:16], scale=math.nan), ds4.Rope(f[1:17])):
        with pytest.raises(ds4.Ds4MoeError):
            call(bad)
    for kw in (dict(q=q[:5]), dict(q=q.bfloat16()), dict(q_out=q.bfloat16()), dict(q=q, q_out=q), dict(q=q[:, :3]),
               dict(q=q, q_out=torch.empty(6, 4, 32, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        call("rope")
    with pytest.raises(ValueError):
        at.append(cache, k, v, t["kv_len"], q=q)
    with pytest.raises(ValueError):
        ds4.Rope(torch.ones(8))
    # outputs over inputs: the 16-bit rows would be read after they are written
    with pytest.raises(ds4.Ds4MoeError):
        call(q=q, q_out=q.view(torch.bfloat16).flatten()[:6 * 256].view(6, 4, 64))
    L = ds4.lib()
    n = ctypes.c_void_p
    args = [at._h, cache.ref, t["rope"].ref, n(q.data_ptr()), 256, None, 256, n(k.data_ptr()), 128, n(v.data_ptr()), 128, 0,
            None, n(t["kv_len"].data_ptr()), 2, 6, None]
    assert L.ds4moe_kv_append_rope(*args) == 1  # queries without a place for them
    args[3] = None
    assert L.ds4moe_kv_append_rope(*args) == 0
    for at_, x in ((2, None), (15, 5), (15, 10 ** 7), (14, 3), (11, 2), (7, None), (8, 100)):
        assert L.ds4moe_kv_append_rope(*[x if i == at_ else y for i, y in enumerate(args)]) == 1, at_
