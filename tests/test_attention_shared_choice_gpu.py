"""Who decides whether a call with shared positions shares, and by what: the host by
the table's capacity, the device by what the arrays hold."""
import pytest
import torch

from tests.attn_ref import DTYPES, attention, gather

pytestmark = pytest.mark.gpu

WIDE = 131072  # positions of a server's longest context


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Batch:
    """Sequences behind `shared` positions, whose pages they have in common, in a
    table as wide as the longest context."""

    def __init__(self, heads, kv, dim, new, page, shared, own, kind="bf16", window=0):
        import deepseek_v4_flash_gb300 as ds4
        self.ds4, self.new = ds4, new
        dt = DTYPES[kind]
        g = torch.Generator().manual_seed(shared + dim + new)
        whole = shared // page
        self.lens = [whole * page + x for x in own]
        counts = [-(-n // page) for n in self.lens]
        self.table = torch.full((len(own), WIDE // page), -1, dtype=torch.int32)
        at = whole
        for b, c in enumerate(counts):
            self.table[b, :whole] = torch.arange(whole)
            self.table[b, whole:c] = torch.arange(at, at + c - whole)
            at += c - whole
        self.k, self.v = [torch.randn(at, page, kv, dim, generator=g).to(dt).cuda() for _ in range(2)]
        self.q = torch.randn(len(own), new, heads, dim, generator=g).to(dt).cuda()
        n = len(own) * new
        self.at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, kind, window, max_seqs=len(own), max_tokens=n, max_shared_tokens=n))
        table = self.table.cuda()
        self.wide, self.tight = ds4.KVCache(self.k, self.v, table), ds4.KVCache(self.k, self.v, table[:, :max(counts)])
        self.len, self.shared = _ints(self.lens), whole * page

    def call(self, cache, *args):
        before = self.at.launch_count()
        out = self.at.decode(cache, self.q, self.len, **dict(zip(("shared_len", "group_start"), args)))
        return out, self.at.launch_count() - before

    def check(self, out):
        for b, n in enumerate(self.lens):
            ref, tol = attention(self.q[b], gather(self.k, self.table, b, n), gather(self.v, self.table, b, n), n - self.new, 0, 0,
                                 self.q.shape[-1] ** -0.5)
            assert ((out[b].double() - ref).abs() <= tol).all(), f"sequence {b}"


SHAPES = [(32, 8, 128, 1, 16), (16, 4, 64, 2, 32), (8, 2, 256, 1, 64), (64, 1, 512, 1, 128)]


@pytest.mark.parametrize("heads,kv,dim,new,page", SHAPES)
def test_a_narrow_view_of_a_wide_table(heads, kv, dim, new, page):
    """max_pages bounds what can be shared: where that would gain nothing the call
    is the plain one, launch for launch and bit for bit."""
    for shared in (600, 0):
        b = Batch(heads, kv, dim, new, page, shared, (5, 30, 64, max(2, new)))
        plain, n = b.call(b.tight)
        out, m = b.call(b.tight, _ints([b.shared]))
        assert m == n and torch.equal(out, plain)
        b.check(out)
        assert b.at.device_error() == 0


@pytest.mark.parametrize("heads,kv,dim,new,page", SHAPES)
def test_a_wide_table(heads, kv, dim, new, page):
    """There the device decides; nothing shared, little, and enough, in one group and
    in two, are the same results."""
    for shared, own in ((0, (700, 3000, 64, max(2, new))), (1501, (5, 200, 64, max(2, new), 90, 33, 1, 150)), (20000, (700, new, 64, 5, 90, 33, 20, 150))):
        own = [max(x, new) for x in own]
        b = Batch(heads, kv, dim, new, page, shared, own)
        half = len(own) // 2
        for args in ((_ints([b.shared]),), (_ints([b.shared, 0]), _ints([0, half, len(own)])), (_ints([0]),)):
            out, _ = b.call(b.wide, *args)
            b.check(out)
        assert b.at.device_error() == 0


def test_flags_of_arrays_that_are_read():
    """shared_len and group_start are read, and their flag raised, where sharing is
    considered: not on a handle with a window, nor where the table is too narrow for it
    to gain, where the call is the plain one whatever they hold."""
    bad = [(_ints([-5]),), (_ints([10 ** 9]),), (_ints([64, 64]), _ints([3, 1, 4])), (_ints([64, 64]), _ints([-1, 2, 99]))]
    for window in (0, 40):
        b = Batch(32, 8, 128, 1, 16, 600, (5, 30, 64, 2), window=window)
        plain, n = b.call(b.tight)
        for args in bad:
            for cache in (b.tight,) if window == 0 else (b.tight, b.wide):
                out, m = b.call(cache, *args)
                assert m == n and torch.equal(out, plain)
        assert b.at.device_error() == 0
    b = Batch(32, 8, 128, 1, 16, 600, (5, 30, 64, 2, 9, 40, 100, 1))
    for args in bad:
        out, _ = b.call(b.wide, *args)
        assert b.at.device_error() == b.ds4.DEVERR_LENGTH
        b.check(out)
