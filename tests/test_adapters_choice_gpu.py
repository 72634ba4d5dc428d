"""Token by token or by tiles: by the adapters that a call uses, not by the slots
that its handle has."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

N_OUT, N_IN, RANK, SLOTS = 1024, 1024, 64, 1000


@pytest.fixture(scope="module")
def many():
    """A handle of many slots, each with an adapter of its own."""
    import deepseek_v4_flash_gb300 as ds4
    g = torch.Generator(device="cuda").manual_seed(1)
    h = ds4.Adapters(N_OUT, N_IN, SLOTS, RANK, max_tokens=4096)
    a = torch.randn(SLOTS, RANK, N_IN, generator=g, device="cuda").bfloat16() / 32
    b = (torch.randn(SLOTS, N_OUT, RANK, generator=g, device="cuda") * 0.3).bfloat16()
    for s in range(SLOTS):
        h.set(s, a[s], b[s], 0.5)
    x = torch.randn(4096, N_IN, generator=g, device="cuda")
    base = torch.randn(4096, N_OUT, generator=g, device="cuda")
    return h, a, b, x, base


def _run(h, x, slots, base, path):
    h.debug_path(path)
    before = h.launch_count()
    y = h.forward(x, slots, torch.empty_like(base), base=base)
    n = h.launch_count() - before
    h.debug_path(0)
    return y, n


def _spread(n, used, slots=SLOTS):
    return ((torch.arange(n, device="cuda") * used // n) * (slots // used)).int()


def _right(y, x, slots, base, a, b):
    """Against 64 bits: 2^-19 of the norm (see test_adapters_sums_gpu.py) of what is added."""
    add = torch.zeros_like(y, dtype=torch.float64)
    for s in set(slots.tolist()):
        if 0 <= s < SLOTS:
            rows = slots == s
            add[rows] = 0.5 * (x[rows].double() @ a[s].double().T) @ b[s].double().T
    off = (y.double() - (base.double() + add)).norm()
    # y is rounded once: 2^-24 of each element
    assert off <= 2.0 ** -19 * add.norm() + 2.0 ** -24 * y.double().norm()


@pytest.mark.parametrize("n,used", [(4096, 1), (4096, 4), (2048, 1), (1024, 3), (3001, 20)])
def test_idle_slots_cost_nothing(many, n, used):
    """Few adapters in a long call: by tiles, however many slots there are."""
    h, a, b, x, base = many
    slots = _spread(n, used)
    slots[::37] = -1
    tiles, _ = _run(h, x[:n], slots, base[:n], 2)
    tokens, _ = _run(h, x[:n], slots, base[:n], 1)
    y, _ = _run(h, x[:n], slots, base[:n], 0)
    assert not torch.equal(tiles, tokens)  # (their roundings tell them apart)
    assert torch.equal(y, tiles)
    _right(y, x[:n], slots, base[:n], a, b)
    assert h.device_error() == 0


@pytest.mark.parametrize("n,used", [(4096, 1000), (1024, 1000), (2048, 500), (700, 700), (64, 1), (64, 64), (1, 1)])
def test_many_adapters_go_token_by_token(many, n, used):
    h, a, b, x, base = many
    slots = _spread(n, used)
    slots[1::41] = -1
    tokens, _ = _run(h, x[:n], slots, base[:n], 1)
    y, _ = _run(h, x[:n], slots, base[:n], 0)
    assert torch.equal(y, tokens)
    _right(y, x[:n], slots, base[:n], a, b)
    assert h.device_error() == 0


def test_one_graph_either_way(many):
    """The choice is made when a captured call runs: from what its slots are then."""
    import deepseek_v4_flash_gb300 as ds4
    h, a, b, x, base = many
    n = 2048
    slots = _spread(n, 2)
    y = torch.empty_like(base[:n])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.forward(x[:n], slots, y, base=base[:n])
    for now, path in ((_spread(n, 2), 2), (_spread(n, 1000), 1), (_spread(n, 5), 2), (torch.full_like(slots, -1), None)):
        now[5], now[77] = SLOTS, -2  # outside: nothing is added
        slots.copy_(now)
        y.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert h.device_error() == ds4.DEVERR_ADAPTER
        if path:
            assert torch.equal(y, _run(h, x[:n], now, base[:n], path)[0])
            assert h.device_error() == ds4.DEVERR_ADAPTER
        _right(y, x[:n], now, base[:n], a, b)
        assert torch.equal(y[5], base[5])
        assert path or torch.equal(y, base[:n])


def test_in_place_and_other_types():
    """The choice on the device with 16-bit inputs, added in place, empty slots."""
    import deepseek_v4_flash_gb300 as ds4
    g = torch.Generator(device="cuda").manual_seed(3)
    h = ds4.Adapters(520, 512, 2000, 100, "fp16", max_tokens=1500)
    a = torch.randn(100, 512, generator=g, device="cuda").half() / 24
    b = (torch.randn(520, 100, generator=g, device="cuda") * 0.3).half()
    for s in range(0, 2000, 2):
        h.set(s, a[:1 + s % 100], b[:, :1 + s % 100].contiguous(), 1.0)
    x = torch.randn(1500, 512, generator=g, device="cuda").half()
    for used in (2, 1500):
        slots = _spread(1500, used, 2000)
        y0 = torch.randn(1500, 520, generator=g, device="cuda")
        got = []
        for path in (0, 1, 2):
            h.debug_path(path)
            got.append(h.forward(x, slots, y0.clone()))
        h.debug_path(0)
        assert torch.equal(got[0], got[2 if used == 2 else 1])
        assert torch.equal(got[0][slots % 2 == 1], y0[slots % 2 == 1])  # odd slots are empty
        assert (got[1] - got[2]).norm() < 2.0 ** -18 * (got[1] - y0).norm() + 2.0 ** -22 * y0.norm()
    assert h.device_error() == 0
