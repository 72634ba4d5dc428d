"""How exact the adapters' sums are, as a whole: the norm of the difference from
64 bits over the norm of the result. (A bound for each element has to allow for
the worst case of every addition and is far above what dropped bits would do.)

Few tokens: fused multiply-adds of products that are exact in 32 bits, rounded to
nearest: a chain of C additions of numbers of random sign is off by some
sqrt(C) 2^-25 of its result, C = 65536 / 8 / 32 + 13 at most (a lane's part, the
lanes, the blocks), and so is the second product: below 2^-20.

Many tokens: an operand is the sum of two numbers of 11 bits, which leaves out
2^-22 of it at most. The tensor cores cut what an accumulator does not hold: an
addition loses up to 2^-23 of the sum so far, 0.36 of it on average (a cut is
uniform, a number lies anywhere between two powers of two), always towards zero, and
a sum of random terms is 2/3 of its last size on average; 37 additions, the most
that go to one accumulator, lose 37 * 0.36 * 2/3 * 2^-23 = 1.06e-6 = 2^-19.8, the
second product of up to 64 additions is a sum of its own. Below 2^-19, as
test_long_sums has it."""
import math

import pytest
import torch

from tests.attn_ref import DTYPES

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "fp32"), ("bf16", "same"), ("fp16", "fp32"), ("fp16", "same")]


def _off(rank, n_in, max_rank, kind, source, path, n=200, n_out=256):
    import deepseek_v4_flash_gb300 as ds4
    dt = DTYPES[kind]
    g = torch.Generator().manual_seed(rank + n_in)
    a = (torch.randn(rank, n_in, generator=g) / math.sqrt(n_in)).to(dt).cuda()
    b = (torch.randn(n_out, rank, generator=g) * 0.3).to(dt).cuda()
    x = torch.randn(n, n_in, generator=g).to(torch.float32 if source == "fp32" else dt).cuda()
    h = ds4.Adapters(n_out, n_in, 2, max_rank, kind, max_tokens=n)
    h.set(1, a, b, 1.0)
    h.debug_path(path)
    y = h.forward(x, torch.ones(n, dtype=torch.int32).cuda(), torch.zeros(n, n_out).cuda())
    ref = (x.double() @ a.double().T) @ b.double().T
    assert h.device_error() == 0
    h.close()
    return float((y.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("kind,source", TYPES)
@pytest.mark.parametrize("rank,n_in,max_rank", [
    (256, 8192, 256), (256, 14336, 256), (256, 16384, 256), (256, 65536, 256), (160, 16384, 160), (130, 8224, 130),
    (128, 28672, 128), (64, 65536, 64), (8, 14336, 256), (8, 65536, 256), (100, 65536, 250)])
def test_wide_inputs_of_any_rank(rank, n_in, max_rank, kind, source):
    """Many tokens: every rank over every width that is accepted, and adapters of
    a small rank on a handle for large ones."""
    off = _off(rank, n_in, max_rank, kind, source, 2)
    print(f"rank {rank} of {max_rank}, {n_in} columns: off by {off:.2e}")
    assert off < 2.0 ** -19


@pytest.mark.parametrize("kind,source", TYPES)
@pytest.mark.parametrize("rank", [1, 16, 64, 65, 128, 129, 200, 256])
@pytest.mark.parametrize("n_in", [1056, 4096, 8192])
def test_the_result_as_a_whole(n_in, rank, kind, source):
    for path, bound in ((1, 2.0 ** -20), (2, 2.0 ** -19)):
        off = _off(rank, n_in, rank, kind, source, path)
        assert off < bound, f"path {path}: off by {off:.2e}"


@pytest.mark.parametrize("rank,n_in", [(256, 65536), (16, 65536), (250, 32)])
def test_few_tokens_over_wide_inputs(rank, n_in):
    for kind, source in TYPES:
        assert _off(rank, n_in, rank, kind, source, 1, n=9) < 2.0 ** -20


def test_infinities_in_wide_inputs():
    """Where a sum is taken in several parts they come out as in one: an infinity
    stays in its row, two of opposite sign are NaN, empty slots add nothing."""
    import deepseek_v4_flash_gb300 as ds4
    n, n_in, n_out, rank = 150, 16384, 64, 200
    a, b = torch.ones(rank, n_in).bfloat16().cuda(), torch.ones(n_out, rank).bfloat16().cuda()
    h = ds4.Adapters(n_out, n_in, 2, 256, max_tokens=n)
    h.set(0, a, b, 0.5)
    h.debug_path(2)
    x = torch.ones(n, n_in).cuda()
    x[3, 5], x[4, n_in - 1], x[5, 0], x[5, n_in - 1] = math.inf, -math.inf, math.inf, -math.inf
    slots = torch.zeros(n, dtype=torch.int32).cuda()
    slots[7], slots[8] = 1, -1
    y = h.forward(x, slots, torch.full((n, n_out), 2.0).cuda())
    assert (y[3] == math.inf).all() and (y[4] == -math.inf).all() and torch.isnan(y[5]).all()
    assert (y[7:9] == 2).all()
    rest = torch.ones(n, dtype=torch.bool)
    rest[[3, 4, 5, 7, 8]] = False
    assert (y[rest.cuda()] == 2 + 0.5 * rank * n_in).all()  # whole numbers below 2^24
    assert h.device_error() == 0
