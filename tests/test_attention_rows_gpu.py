"""Row bounds (cu_q) that are out of order or outside the call's rows: they are
brought into [0, n_tok] and raised to the largest before them, so that
sequences never share a row, and DS4MOE_DEVERR_LENGTH is raised."""
import math
import random

import pytest
import torch

from tests.attn_ref import DTYPES, attention, gather, paged, to_cuda

pytestmark = pytest.mark.gpu


def _clean(cu, n_tok):
    out, top = [], 0
    for c in cu:
        top = max(top, min(max(c, 0), n_tok))
        out.append(top)
    return out


def _bounds(kind, n_seq, T):
    rng = random.Random(n_seq)
    if kind == "repeat":  # every second sequence would have all rows
        return [T * (i % 2) for i in range(n_seq + 1)]
    if kind == "outside":
        return [-5] + sorted(rng.randint(0, T) for _ in range(n_seq - 1)) + [T + 1000]
    cu = [0] + sorted(rng.randint(0, T) for _ in range(n_seq - 1)) + [T]
    for _ in range(max(1, n_seq // 8)):  # neighbours swapped, some pairs far apart
        i, j = rng.randrange(n_seq + 1), rng.randrange(n_seq + 1)
        cu[i], cu[j] = cu[j], cu[i]
    cu[n_seq // 2], cu[n_seq // 2 + 1] = T - 3, 2 ** 31 - 1
    return cu


def _setup(kind, n_seq, T, kv, dim, seed):
    cu = _bounds(kind, n_seq, T)
    clean = _clean(cu, T)
    assert clean != cu
    lens = [clean[b + 1] - clean[b] + (7 * b) % 23 for b in range(n_seq)]
    k, v, table = paged(lens, 16, kv, dim, torch.bfloat16, seed)
    return cu, clean, lens, *to_cuda(k, v), table


@pytest.mark.parametrize("kind", ["repeat", "outside", "swapped"])
@pytest.mark.parametrize("n_seq", [5, 32, 33, 64, 1500])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (8, 1, 256), (64, 1, 512)])
def test_prefill_rows_out_of_order(kind, n_seq, heads, kv, dim):
    """Calls with a planning launch (more than 32 sequences) and without; a
    handle whose workspace is no larger than the call needs."""
    import deepseek_v4_flash_gb300 as ds4
    T = 600
    cu, clean, lens, kd, vd, table = _setup(kind, n_seq, T, kv, dim, 3)
    q = torch.randn(T, heads, dim, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, max_seqs=n_seq, max_tokens=T))
    cache = ds4.KVCache(kd, vd, table.cuda())
    length = torch.tensor(lens, dtype=torch.int32).cuda()
    good = at.prefill(cache, q, torch.tensor(clean, dtype=torch.int32).cuda(), length, out=torch.full_like(q, math.nan))
    assert at.device_error() == 0
    got = at.prefill(cache, q, torch.tensor(cu, dtype=torch.int32).cuda(), length, out=torch.full_like(q, math.nan))
    assert at.device_error() == ds4.DEVERR_LENGTH and at.device_error() == 0
    assert torch.equal(got.view(torch.int16), good.view(torch.int16))
    for b in range(n_seq):
        a, e = clean[b], clean[b + 1]
        if a == e:
            continue
        ref, tol = attention(q[a:e], gather(kd, table, b, lens[b]), gather(vd, table, b, lens[b]), lens[b] - (e - a), 0,
                             0, dim ** -0.5)
        assert ((got[a:e].double() - ref).abs() <= tol).all()
    # rows of no sequence are left as they are
    assert torch.isnan(got[:clean[0]]).all() and torch.isnan(got[clean[-1]:]).all()


@pytest.mark.parametrize("kind", ["repeat", "outside", "swapped"])
@pytest.mark.parametrize("n_seq", [5, 64, 1023, 1024, 1025, 2600])
@pytest.mark.parametrize("source", [torch.float32, torch.bfloat16])
def test_append_rows_out_of_order(kind, n_seq, source):
    """The append takes the same bounds as the attention calls: the same rows
    of the same sequences, and the flag. More than 1024 sequences: another
    launch."""
    import deepseek_v4_flash_gb300 as ds4
    T, kv, dim = 900, 2, 64
    cu = _bounds(kind, n_seq, T)
    clean = _clean(cu, T)
    lens = [clean[b + 1] - clean[b] + (7 * b) % 23 for b in range(n_seq)]
    k, v, table = paged(lens, 16, kv, dim, torch.bfloat16, 5, fill=0.25)
    kd, vd = to_cuda(k, v)
    g = torch.Generator().manual_seed(9)
    kn, vn = torch.randn(T, kv, dim, generator=g).to(source), torch.randn(T, kv, dim, generator=g).to(source)
    at = ds4.Attention(ds4.AttentionDesc(kv, kv, dim, max_seqs=n_seq, max_tokens=T))
    at.append(ds4.KVCache(kd, vd, table.cuda()), kn.cuda(), vn.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
              cu_q=torch.tensor(cu, dtype=torch.int32).cuda())
    assert at.device_error() == ds4.DEVERR_LENGTH and at.device_error() == 0
    for b in range(n_seq):
        a, e = clean[b], clean[b + 1]
        for j in range(e - a):
            pos = lens[b] - (e - a) + j
            k[table[b, pos // 16], pos % 16] = kn[a + j].bfloat16()
            v[table[b, pos // 16], pos % 16] = vn[a + j].bfloat16()
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


@pytest.mark.parametrize("n_seq", [1, 70, 1024, 1025, 2600])
def test_append_many_sequences(n_seq):
    """Ascending bounds, empty sequences among them, and rows of no sequence
    at either end: no flag."""
    import deepseek_v4_flash_gb300 as ds4
    T, kv, dim = 900, 1, 64
    rng = random.Random(n_seq)
    cu = sorted(rng.randint(11, T - 13) for _ in range(n_seq + 1))
    lens = [cu[b + 1] - cu[b] + b % 5 for b in range(n_seq)]
    k, v, table = paged(lens, 16, kv, dim, torch.bfloat16, 5, fill=0.25)
    kd, vd = to_cuda(k, v)
    kn = torch.randn(T, kv, dim, generator=torch.Generator().manual_seed(2))
    at = ds4.Attention(ds4.AttentionDesc(kv, kv, dim, max_seqs=n_seq, max_tokens=T))
    at.append(ds4.KVCache(kd, vd, table.cuda()), kn.cuda(), -kn.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
              cu_q=torch.tensor(cu, dtype=torch.int32).cuda())
    assert at.device_error() == 0
    for b in range(n_seq):
        for j in range(cu[b + 1] - cu[b]):
            pos = b % 5 + j
            k[table[b, pos // 16], pos % 16] = kn[cu[b] + j].bfloat16()
            v[table[b, pos // 16], pos % 16] = -kn[cu[b] + j].bfloat16()
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)
