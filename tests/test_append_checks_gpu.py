"""Shapes that an append refuses."""
import pytest
import torch

from tests.attn_ref import paged, to_cuda

pytestmark = pytest.mark.gpu


def test_rows_of_other_sequences_than_the_lengths():
    """[2 sequences, 3 tokens] with three lengths: not the six rows as two
    tokens of three sequences."""
    import deepseek_v4_flash_gb300 as ds4
    k, v, table = paged([20, 20, 20], 16, 2, 64, torch.bfloat16, 5, fill=0.0)
    kd, vd = to_cuda(k, v)
    at = ds4.Attention(ds4.AttentionDesc(2, 2, 64, max_seqs=3, max_tokens=6))
    cache = ds4.KVCache(kd, vd, table.cuda())
    new = torch.randn(2, 3, 2, 64).cuda()
    length = torch.tensor([20, 20, 20], dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        at.append(cache, new, new, length)
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)
    at.append(cache, new.view(6, 2, 64), None, length)  # rows without that claim: two of each
    at.append(cache, new.view(3, 2, 2, 64), None, length)
    assert at.device_error() == 0
