"""Low-rank adapters (ds4moe_adapters_*) against their formula in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests.attn_ref import DTYPES

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


def _weights(ranks, n_out, n_in, dt, seed):
    g = torch.Generator().manual_seed(seed)
    a = [(torch.randn(r, n_in, generator=g) / math.sqrt(n_in)).to(dt) for r in ranks]
    b = [(torch.randn(n_out, r, generator=g) * 0.3).to(dt) for r in ranks]
    return a, b, [0.25 + 1.5 * i for i in range(len(ranks))]


def _handle(ranks, n_out, n_in, kind, n_tok, seed, max_rank=None, path=None):
    a, b, s = _weights(ranks, n_out, n_in, DTYPES[kind], seed)
    h = _ds4().Adapters(n_out, n_in, len(ranks), max_rank or max(ranks), kind, max_tokens=n_tok)
    for i in range(len(ranks)):
        h.set(i, a[i].cuda(), b[i].cuda(), s[i])
    # few tokens one by one, more by tiles, whatever the automatic choice
    h.debug_path(path or (1 if n_tok <= 64 else 2))
    return h, a, b, s


def _expect(x, slots, base, a, b, s):
    """y in 64 bits and the error that 32-bit sums may make.

    h = A x: an operand is taken as its leading 11 bits and the leading 11 of the
    rest, which is below 2^-10 of it, so 2^-20 of it is left out; at most n_in / 4
    additions of partial sums, each cut (not rounded) to 24 bits: the error is
    below (2^-20 + n_in / 4 2^-23) of sum |a x|; y likewise over the rank, plus
    what h's error brings, plus a rounding of scale h and of y."""
    y, tol = base.double().clone(), 2.0 ** -23 * base.double().abs()
    for i in set(slots.tolist()):
        if not 0 <= i < len(a):
            continue
        rows = slots == i
        xx, A, B = x[rows].double(), a[i].double(), b[i].double()
        h, hs = xx @ A.T, xx.abs() @ A.abs().T
        n_in, r = A.shape[1], A.shape[0]
        eh = (2.0 ** -20 + n_in / 4 * 2.0 ** -23) * hs
        size = hs @ B.abs().T
        y[rows] += s[i] * (h @ B.T)
        tol[rows] += abs(s[i]) * (eh @ B.abs().T + (2.0 ** -20 + (r / 4 + 8) * 2.0 ** -23) * size)
    return y, tol + 1e-30


def _close(got, ref, tol, what=""):
    got = got.double().cpu()
    same = torch.isnan(got) & torch.isnan(ref) | (got == ref)
    over = torch.where(same, -1.0, (got - ref).abs() - tol)
    assert (over <= 0).all(), f"{what}: {int((~(over <= 0)).sum())} of {got.numel()} off, worst " \
                              f"{float((got - ref).abs().nan_to_num().max())}"


def _run(kind, source, n_out, n_in, ranks, slots, seed=0, max_rank=None, path=None):
    n = len(slots)
    h, a, b, s = _handle(ranks, n_out, n_in, kind, n, seed, max_rank, path)
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(n, n_in, generator=g).to(torch.float32 if source == "fp32" else DTYPES[kind])
    base = torch.randn(n, n_out, generator=g)
    slots = torch.tensor(slots, dtype=torch.int32)
    ref, tol = _expect(x, slots, base, a, b, s)
    xd, sd, bd = x.cuda(), slots.cuda(), base.cuda()
    y = torch.full((n, n_out), math.nan).cuda()
    assert h.forward(xd, sd, y, base=bd) is y
    _close(y, ref, tol, "from base")
    again = torch.empty_like(y)
    h.forward(xd, sd, again, base=bd)
    assert torch.equal(y, again), "two calls differ"
    h.forward(xd, sd, bd)
    assert torch.equal(y, bd), "added in place differs"
    assert h.device_error() == 0
    h.close()


SHAPES = [(32, 32), (1, 64), (7, 96), (256, 256), (1027, 416), (4096, 4096), (130, 8192)]


@pytest.mark.parametrize("kind,source", [("bf16", "fp32"), ("bf16", "same"), ("fp16", "fp32"), ("fp16", "same")])
@pytest.mark.parametrize("n_out,n_in", SHAPES)
def test_few_tokens(kind, source, n_out, n_in):
    """One to 64 tokens, ranks of every remainder, tokens without an adapter."""
    ranks = [1, 5, 8, 16, 33, 64]
    _run(kind, source, n_out, n_in, ranks, [3], 1)
    _run(kind, source, n_out, n_in, ranks, [-1, 0, 1, 2, 3, 4, 5, 5, -1], 2)
    _run(kind, source, n_out, n_in, ranks, [(5 * t) % 7 - 1 for t in range(64)], 3, max_rank=100)


@pytest.mark.parametrize("kind,source", [("bf16", "fp32"), ("bf16", "same"), ("fp16", "fp32"), ("fp16", "same")])
@pytest.mark.parametrize("n_out,n_in", SHAPES)
def test_many_tokens(kind, source, n_out, n_in):
    """Runs of one adapter, adapters in no order, tiles that end inside a run."""
    ranks = [16, 1, 40, 64]
    _run(kind, source, n_out, n_in, ranks, [0] * 65, 4)
    _run(kind, source, n_out, n_in, ranks, [2] * 128 + [1] * 129 + [-1] * 40 + [3] * 3, 5)
    _run(kind, source, n_out, n_in, ranks, [(7 * t) % 5 - 1 for t in range(777)], 6, max_rank=65)


@pytest.mark.parametrize("rank", [31, 32, 127, 128, 200, 255, 256])
@pytest.mark.parametrize("n", [3, 300])
def test_ranks(rank, n):
    _run("bf16", "fp32", 384, 1056, [rank, 2], [t % 2 for t in range(n)], rank)


@pytest.mark.parametrize("rank,n_in", [(100, 8192), (250, 4096), (64, 16384), (16, 65536)])
def test_long_sums(rank, n_in):
    """Sums over so many columns stay as exact as 32-bit ones: the result as a
    whole is off by less than 2^-19 (the operands' split alone may take 2^-20)."""
    n, n_out = 200, 256
    h, a, b, s = _handle([rank], n_out, n_in, "bf16", n, 19)
    x, base = torch.randn(n, n_in), torch.zeros(n, n_out)
    slots = torch.zeros(n, dtype=torch.int32)
    y = h.forward(x.cuda(), slots.cuda(), torch.empty(n, n_out).cuda(), base=base.cuda())
    ref, tol = _expect(x, slots, base, a, b, s)
    _close(y, ref, tol)
    off = float((y.double().cpu() - ref).norm() / ref.norm())
    print(f"rank {rank}, {n_in} columns: off by {off:.2e}")
    assert off < 2.0 ** -19


def test_many_slots():
    """A batch of more adapters than a warp has lanes, most with one token."""
    ranks = [1 + (3 * i) % 17 for i in range(300)]
    _run("bf16", "fp32", 100, 128, ranks, [(17 * t) % 300 for t in range(40)], 7)
    _run("bf16", "fp32", 100, 128, ranks, [(17 * t) % 300 for t in range(500)], 8)


@pytest.mark.parametrize("n", [1, 2, 63, 65, 130, 700])
def test_either_way_for_any_number_of_tokens(n):
    for path in (1, 2):
        _run("bf16", "fp32", 260, 352, [33, 3, 9], [(5 * t) % 4 - 1 for t in range(n)], n, path=path)


def test_the_automatic_choice():
    """One launch for a step, three for a prompt, and the same results but for roundings."""
    n = 900
    h, a, b, s = _handle([16, 8], 512, 512, "bf16", n, 18)
    h.debug_path(0)
    x, base = torch.randn(n, 512), torch.randn(n, 512)
    for m, launches in ((1, 1), (64, 1), (900, 3)):
        slots = torch.tensor([t % 3 - 1 for t in range(m)], dtype=torch.int32)
        before = h.launch_count()
        y = h.forward(x[:m].cuda(), slots.cuda(), torch.empty(m, 512).cuda(), base=base[:m].cuda())
        assert h.launch_count() - before == launches
        ref, tol = _expect(x[:m], slots, base[:m], a, b, s)
        _close(y, ref, tol)
    with pytest.raises(_ds4().Ds4MoeError):
        h.debug_path(3)


def test_long_prompt():
    """More tiles than clusters run at once, and one that all blocks share."""
    _run("bf16", "fp32", 512, 1024, [64, 16], [0] * 9000 + [1] * 3001, 9)
    _run("fp16", "same", 512, 1024, [64, 16], [0] * 40000 + [1] * 25000, 10)


def test_set_replaces_and_clear_empties():
    ds4 = _ds4()
    n_out, n_in = 160, 256
    g = torch.Generator().manual_seed(11)
    h = ds4.Adapters(n_out, n_in, 3, 40, "bf16", max_tokens=200)
    for n in (4, 200):
        h.debug_path(1 if n == 4 else 2)
        x = torch.randn(n, n_in, generator=g).cuda()
        y = torch.randn(n, n_out, generator=g).cuda()
        slots = torch.tensor([t % 3 for t in range(n)], dtype=torch.int32).cuda()
        for i in range(3):
            h.clear(i)
        before = y.clone()
        h.forward(x, slots, y)
        assert torch.equal(y, before)  # empty slots add nothing
        # a longer adapter, then a shorter one in the same place: nothing is left of the first
        for rank in (40, 3):
            a, b, s = _weights([rank], n_out, n_in, torch.bfloat16, rank)
            h.set(1, a[0].cuda(), b[0].cuda(), 2.0)
            out = torch.empty_like(y)
            h.forward(x, slots, out, base=y)
            ref, tol = _expect(x.cpu(), torch.where(slots == 1, 0, -1).cpu(), y.cpu(), a, b, [2.0])
            _close(out, ref, tol, f"rank {rank}")
        out = torch.empty_like(y)
        h.forward(x, slots, out, base=y)
        h.clear(1)
        h.forward(x, slots, out, base=y)
        assert torch.equal(out, y)
    assert h.device_error() == 0


@pytest.mark.parametrize("n", [5, 300])
def test_slots_that_there_are_not(n):
    ds4 = _ds4()
    h, a, b, s = _handle([8, 4], 96, 128, "bf16", n, 12)
    x, base = torch.randn(n, 128), torch.randn(n, 96)
    slots = torch.tensor([[0, 2, 1, -2, 2 ** 31 - 1][t % 5] for t in range(n)], dtype=torch.int32)
    y = torch.empty(n, 96).cuda()
    h.forward(x.cuda(), slots.cuda(), y, base=base.cuda())
    ref, tol = _expect(x, slots, base, a, b, s)
    _close(y, ref, tol)
    assert torch.equal(y[1].cpu(), base[1])
    assert h.device_error() == ds4.DEVERR_ADAPTER and h.device_error() == 0


@pytest.mark.parametrize("n", [6, 200])
def test_numbers_that_are_not_finite(n):
    """They stay in their rows; an infinity comes out as the formula has it."""
    h, a, b, s = _handle([7, 16], 96, 128, "bf16", n, 13)
    x, base = torch.randn(n, 128), torch.randn(n, 96)
    a[0].abs_()
    b[0].abs_()
    h.set(0, a[0].cuda(), b[0].cuda(), s[0])
    slots = torch.tensor([t % 2 for t in range(n)], dtype=torch.int32)
    x[0, 5], x[2, 7], x[3, 0], base[5, 5] = math.inf, -math.inf, math.nan, math.inf
    x[4] *= 1e30
    y = torch.empty(n, 96).cuda()
    h.forward(x.cuda(), slots.cuda(), y, base=base.cuda())
    assert (y[0] == math.inf).all() and (y[2] == -math.inf).all() and torch.isnan(y[3]).all() and y[5, 5] == math.inf
    rest = [t for t in range(n) if t not in (0, 2, 3)]
    ref, tol = _expect(x[rest], slots[rest], base[rest], a, b, s)
    _close(y[rest], ref, torch.where(torch.isfinite(ref), tol, 0.0))


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("where", ["a", "b", "x"])
@pytest.mark.parametrize("rank", [1, 40, 200])
def test_infinities_beside_short_numbers(rank, where, kind, path):
    """Operands of few bits, of which an infinity is one: the others' products
    are exact, and what they leave out is 0, not 0 times infinity."""
    dt, n_in, n_out = DTYPES[kind], 64, 140
    a, b = torch.ones(rank, n_in, dtype=dt), torch.ones(n_out, rank, dtype=dt)
    x, base = torch.ones(130, n_in), torch.zeros(130, n_out)
    want = torch.full((130, n_out), float(n_in * rank))
    if where == "a":
        a[rank - 1, 3] = math.inf
        want[:] = math.inf
    elif where == "b":
        b[7, rank - 1], b[131, 0] = math.inf, -math.inf
        want[:, 7], want[:, 131] = math.inf, -math.inf
    else:
        x[5, 63], x[129, 0] = math.inf, -math.inf
        want[5], want[129] = math.inf, -math.inf
    h = _ds4().Adapters(n_out, n_in, 1, rank, kind, max_tokens=130)
    h.set(0, a.cuda(), b.cuda(), 1.0)
    h.debug_path(path)
    y = torch.empty(130, n_out).cuda()
    h.forward(x.cuda(), torch.zeros(130, dtype=torch.int32).cuda(), y, base=base.cuda())
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("n", [9, 150])
def test_columns_of_one_matrix(n):
    """x, base and y as columns of the same rows."""
    h, a, b, s = _handle([8, 20], 64, 96, "fp16", n, 21)
    rows = torch.randn(n, 240).cuda()
    before = rows.cpu()
    x, base, y = rows[:, :96], rows[:, 100:164], rows[:, 172:236]
    slots = torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32)
    h.forward(x, slots.cuda(), y, base=base)
    ref, tol = _expect(before[:, :96], slots, before[:, 100:164], a, b, s)
    _close(y, ref, tol)
    before[:, 172:236] = y.cpu()
    assert torch.equal(rows.cpu(), before)
    for bad in (rows[:, 95:159], rows[:, 163:227]):
        with pytest.raises(_ds4().Ds4MoeError):
            h.forward(x, slots.cuda(), bad, base=base)


@pytest.mark.parametrize("n", [9, 150])
def test_strided_rows_and_other_rows_left_alone(n):
    """x, base and y as parts of wider rows, y not 16-byte aligned."""
    for n_out, wide, off in ((64, 200, 8), (64, 131, 1), (33, 77, 3)):
        h, a, b, s = _handle([8, 20], n_out, 96, "fp16", n, 14)
        x, base = torch.randn(n, 400).cuda(), torch.randn(n + 2, wide).cuda()
        y = torch.full((n + 2, wide), 3.0).cuda()
        slots = torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32).cuda()
        got = h.forward(x[:, 100:196], slots, y[1:-1, off:off + n_out], base=base[1:-1, off:off + n_out])
        ref, tol = _expect(x[:, 100:196].cpu(), slots.cpu(), base[1:-1, off:off + n_out].cpu(), a, b, s)
        _close(got, ref, tol)
        rest = torch.ones_like(y, dtype=torch.bool)
        rest[1:-1, off:off + n_out] = False
        assert (y[rest] == 3).all()


@pytest.mark.parametrize("n", [3, 200])
def test_captured_and_on_another_stream(n):
    h, a, b, s = _handle([8, 20], 128, 256, "bf16", n, 15)
    x, base = torch.randn(n, 256), torch.randn(n, 128)
    slots = torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32)
    xd, bd, sd, y = x.cuda(), base.cuda(), slots.cuda(), torch.empty(n, 128).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h.forward(xd, sd, y, base=bd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref, tol = _expect(x, slots, base, a, b, s)
    _close(y, ref, tol)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        h.forward(xd, sd, y, base=bd)
    slots = slots.roll(1)
    sd.copy_(slots)
    xd.copy_(x.flip(0))
    h.set(0, a[0].cuda(), b[0].cuda(), -1.0)  # the graph uses what the slot holds when it runs
    g.replay()
    torch.cuda.synchronize()
    ref, tol = _expect(x.flip(0), slots, base, a, b, [-1.0, s[1]])
    _close(y, ref, tol)


@pytest.mark.parametrize("n", [1, 4, 70])
def test_beside_the_dense_product(n):
    """Dense.forward(adapters=): the product's own bits, then the adapters."""
    import synth
    ds4 = _ds4()
    n_out, n_in = 96, 128
    w = torch.from_numpy(synth.gen_q8_matrix(3, n_out, n_in, 0.05)).cuda()
    dense = ds4.Dense(n_out, n_in, w, max_tokens=n)
    h, a, b, s = _handle([8, 20], n_out, n_in, "bf16", n, 16)
    x = torch.from_numpy(np.ascontiguousarray(synth.gen_dense_x(4, n, n_in))).cuda()
    slots = torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32).cuda()
    plain = dense.forward(x)
    y = dense.forward(x, adapters=h, slots=slots)
    both = torch.empty_like(y)
    h.forward(x, slots, both, base=plain)
    assert torch.equal(y, both)
    ref, tol = _expect(x.cpu(), slots.cpu(), plain.cpu(), a, b, s)
    _close(y, ref, tol)
    for kw in (dict(slots=slots), dict(adapters=h), dict(adapters=h, slots=slots[:0]), dict(adapters=h, slots=slots.long())):
        with pytest.raises(ValueError):
            dense.forward(x, **kw)
    other = ds4.Adapters(n_out, n_in + 32, 1, 4)
    with pytest.raises(ValueError):
        dense.forward(x, adapters=other, slots=slots)


def test_refusals():
    ds4 = _ds4()
    h, a, b, s = _handle([8, 20], 64, 96, "bf16", 10, 17)
    x, y, slots = torch.randn(10, 96).cuda(), torch.randn(10, 64).cuda(), torch.zeros(10, dtype=torch.int32).cuda()
    ad, bd = a[0].cuda(), b[0].cuda()
    for args in ((2, ad, bd), (-1, ad, bd), (0, ad, bd, math.nan), (0, ad, bd, math.inf)):
        with pytest.raises(ds4.Ds4MoeError):
            h.set(*args)
    for args in ((0, ad.float(), bd), (0, ad.half(), bd.half()), (0, ad, bd[:, :4]), (0, ad[:, :64], bd), (0, ad.T, bd.T), (0, a[0], b[0])):
        with pytest.raises(ValueError):
            h.set(*args)
    with pytest.raises(ds4.Ds4MoeError):
        h.set(0, torch.zeros(21, 96).bfloat16().cuda(), torch.zeros(64, 21).bfloat16().cuda())
    for args in ((x[:, :64], slots, y), (x, slots[:9], y), (x, slots.long(), y), (x, slots, y[:9]), (x, slots, y.double()),
                 (x.half(), slots, y), (x.cpu(), slots, y), (x, slots, y, y[:, :32])):
        with pytest.raises(ValueError):
            h.forward(*args)
    wide = torch.randn(11, 96).cuda()
    with pytest.raises(ds4.Ds4MoeError):
        h.forward(wide, torch.zeros(11, dtype=torch.int32).cuda(), torch.zeros(11, 64).cuda())  # more than max_tokens
    with pytest.raises(ds4.Ds4MoeError):
        h.forward(torch.randn(10, 101).cuda()[:, 1:97], slots, y)  # rows that are not aligned
    both = torch.randn(20, 64).cuda()
    with pytest.raises(ds4.Ds4MoeError):
        h.forward(x, slots, both[:10], base=both[1:11])
    with pytest.raises(ds4.Ds4MoeError):
        h.forward(wide.flatten()[:960].view(10, 96), slots, wide.flatten()[:640].view(10, 64))
    before = y.clone()
    h.forward(x[:0], slots[:0], y[:0])
    assert torch.equal(before, y)
    L, n = ds4.lib(), ctypes.c_void_p
    good = [h._h, n(x.data_ptr()), 96, 0, n(slots.data_ptr()), 10, None, 0, n(y.data_ptr()), 64, None]
    for at, bad in ((1, None), (2, 95), (2, 97), (3, 2), (3, 7), (4, None), (5, -1), (5, 11), (8, None), (9, 63)):
        assert L.ds4moe_adapters_forward(*[bad if i == at else v for i, v in enumerate(good)]) == 1, (at, bad)
    assert L.ds4moe_adapters_forward(*good) == 0 and h.device_error() == 0
    assert h.launch_count() >= 1 and h.device_bytes() > 2 * 2 * 20 * 160
