"""Values that are not finite under weights of almost nothing or nothing: a call
with shared positions gives them as the call without does. A position that a row
sees has a weight above zero, however small, or exactly zero where its score is
-infinity, and zero times NaN is NaN; only a row without any score above
-infinity is zero, whatever its values."""
import math

import pytest
import torch

from tests.attn_ref import DTYPES

pytestmark = pytest.mark.gpu

PAGE = 16
SHAPES = [(8, 2, 128, 1), (8, 2, 128, 2), (6, 2, 64, 3), (8, 8, 64, 1), (8, 1, 256, 2), (64, 1, 512, 1), (64, 1, 512, 4)]
LENGTHS = [(256, 44), (20000, 44), (256, 5000), (20000, 5000)]  # one block and many for the shared, the own positions


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Case:
    """Three sequences behind `shared` positions (whole pages)."""

    def __init__(self, heads, kv, dim, new, shared, own, kind):
        import deepseek_v4_flash_gb300 as ds4
        g = torch.Generator().manual_seed(shared + own + dim)
        self.first, each, n = shared // PAGE, -(-own // PAGE), 3
        shape = (self.first + n * each, PAGE, kv, dim)
        self.k = torch.randn(shape, generator=g).to(DTYPES[kind]).cuda()
        self.v = torch.randn(shape, generator=g).to(DTYPES[kind]).cuda()
        table = [list(range(self.first)) + list(range(self.first + each * b, self.first + each * (b + 1))) for b in range(n)]
        self.q = torch.randn(n, new, heads, dim, generator=g).to(DTYPES[kind]).cuda().abs() + 0.25
        self.at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, max_seqs=n, max_tokens=n * new, max_shared_tokens=n * new))
        self.at.debug_share()
        self.cache, self.len = ds4.KVCache(self.k, self.v, _ints(table)), _ints([shared + own] * n)
        self.shared, self.group = _ints([shared]), heads // kv

    def both(self):
        plain = self.at.decode(self.cache, self.q, self.len)
        out = self.at.decode(self.cache, self.q, self.len, shared_len=self.shared)
        assert self.at.device_error() == 0
        return plain, out


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shared,own", LENGTHS)
@pytest.mark.parametrize("heads,kv,dim,new", SHAPES)
def test_under_weights_of_almost_nothing(heads, kv, dim, new, shared, own, kind):
    """One element of a value, of a position whose weight is below 2^-149."""
    c = Case(heads, kv, dim, new, shared, own, kind)
    for low, high, page in ((slice(None, c.first), slice(c.first, None), 2), (slice(c.first, None), slice(None, c.first), c.first)):
        c.k[low], c.k[high] = -30.0, 30.0  # scores of -30 and 30 times dim^0.5 (0.25 + |q|): more than 200 apart
        plain, clean = c.both()
        assert torch.isfinite(clean.float()).all()
        keep = c.v[page, 3].clone()
        for bad in (math.nan, math.inf):
            c.v[page, 3, 0, 5] = bad
            plain, out = c.both()
            want = torch.zeros_like(out, dtype=torch.bool)
            rows = slice(None) if page == 2 else slice(0, 1)  # the shared one of all sequences, the own one of the first
            want[rows, :, :c.group, 5] = True
            assert torch.equal(torch.isnan(plain), want)
            assert torch.equal(torch.isnan(out), want)
            assert torch.equal(out[~want], clean[~want])
            c.v[page, 3] = keep


@pytest.mark.parametrize("shared,own", LENGTHS)
@pytest.mark.parametrize("heads,kv,dim,new", SHAPES)
def test_under_weights_of_nothing(heads, kv, dim, new, shared, own):
    """Scores of -infinity: of all shared positions, of all own ones, of both."""
    c = Case(heads, kv, dim, new, shared, own, "bf16")
    kk = c.k.clone()
    for low, page in ((slice(None, c.first), 2), (slice(c.first, None), c.first)):
        c.k.copy_(kk)
        c.k[low] = -math.inf
        plain, clean = c.both()
        assert torch.isfinite(clean.float()).all()
        keep = c.v[page, 3].clone()
        c.v[page, 3, 0, 5] = math.nan
        plain, out = c.both()
        want = torch.zeros_like(out, dtype=torch.bool)
        rows = slice(None) if page == 2 else slice(0, 1)
        want[rows, :, :c.group, 5] = True
        assert torch.equal(torch.isnan(plain), want)
        assert torch.equal(torch.isnan(out), want)
        assert torch.equal(out[~want], clean[~want])
        c.k[:] = -math.inf
        plain, out = c.both()
        assert (plain == 0).all() and (out == 0).all()
        c.v[page, 3] = keep


@pytest.mark.parametrize("shared,own", LENGTHS)
@pytest.mark.parametrize("heads,kv,dim,new", [s for s in SHAPES if s[3] > 1])
def test_rows_before_the_value_stay_finite(heads, kv, dim, new, shared, own):
    """The value of the last new token: seen by its row alone. Also where the first
    row sees the shared positions alone, and has no own one."""
    c = Case(heads, kv, dim, new, shared, own, "bf16")
    for mine in (own, new, new - 1):
        c.len.fill_(shared + mine)
        plain, clean = c.both()
        at = mine - 1
        for bad in (math.nan, math.inf):
            keep = c.v[c.first + at // PAGE, at % PAGE].clone()
            c.v[c.first + at // PAGE, at % PAGE] = bad
            plain, out = c.both()
            assert (~torch.isfinite(out[0, -1].float())).all()
            assert torch.isfinite(out[0, :-1].float()).all() and torch.equal(out[1:], clean[1:])
            assert torch.allclose(out[0, :-1].float(), clean[0, :-1].float(), atol=2.0 ** -6, rtol=2.0 ** -6)
            c.v[c.first + at // PAGE, at % PAGE] = keep
