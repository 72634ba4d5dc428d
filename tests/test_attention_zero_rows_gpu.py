"""Rows that see positions, but no score above -infinity."""
import math

import pytest
import torch

from tests.attn_ref import paged, to_cuda

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


@pytest.mark.parametrize("heads,kv,dim,new", [(8, 2, 128, 1), (8, 2, 128, 3), (4, 4, 64, 1), (4, 1, 256, 2), (16, 1, 512, 1),
                                              (64, 1, 512, 4)])
def test_no_score_above_minus_infinity(heads, kv, dim, new):
    """Every visible score is -infinity: zeros, whatever the values hold. One
    finite score among them: its value."""
    ds4 = _ds4()
    n = 700
    k, v, table = paged([n], 32, kv, dim, torch.bfloat16, 3)
    for c in range(-(-n // 32)):
        rows = min(32, n - 32 * c)
        k[table[0, c], :rows] = 0
        k[table[0, c], :rows, :, 0] = -math.inf
        v[table[0, c], :rows, :, 1] = math.nan
    kd, vd = to_cuda(k, v)
    q = torch.zeros(1, new, heads, dim, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    length, cu = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, new], dtype=torch.int32).cuda()
    at = ds4.Attention(ds4.AttentionDesc(heads, kv, dim, max_tokens=new))
    cache = ds4.KVCache(kd, vd, table.cuda())
    assert (at.decode(cache, q.cuda(), length) == 0).all()
    assert (at.prefill(cache, q[0].cuda(), cu, length) == 0).all()
    k[table[0, 2], 5, :, 0] = 1.0
    v[table[0, 2], 5] = 0.75
    for c in range(-(-n // 32)):  # 0 x NaN would be NaN
        v[table[0, c], :min(32, n - 32 * c), :, 1] = 0.75
    kd, vd = to_cuda(k, v)
    cache = ds4.KVCache(kd, vd, table.cuda())
    assert (at.decode(cache, q.cuda(), length) == 0.75).all()
    assert (at.prefill(cache, q[0].cuda(), cu, length) == 0.75).all()
    assert at.device_error() == 0
