"""Verification with probabilities outside [0, 1] and NaN: clamped, NaN as 0,
where a draft is accepted as well as where a token is drawn."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,q,u,accepted", [
    (1.5, 2.0, 0.9, True),              # 0.9 < 1
    (0.9, 2.0, 0.6, True),              # 0.6 < 0.9
    (-1.0, -2.0, 0.9, False),           # 0 < 0
    (-1.0, 0.0, 0.9, False),
    (0.5, math.nan, 0.9, True),         # 0 < 0.5
    (math.nan, 0.5, 0.0, False),        # 0 < 0
    (math.nan, math.nan, 0.5, False),
    (math.inf, math.inf, 0.99, True),   # 0.99 < 1
    (0.5, math.inf, 0.5, False),        # 0.5 < 0.5
    (0.5, -math.inf, 0.99, True),
    (1e-30, 1.0, 0.0, True),
    (0.25, 0.5, 0.5, False),            # equality is not below
])
def test_acceptance_clamps(p, q, u, accepted):
    import deepseek_v4_flash_gb300 as ds4
    V = 7
    target, draft = torch.zeros(1, 2, V), torch.zeros(1, 1, V)
    target[0, :, 4] = 1.0           # what is drawn where nothing else has mass
    target[0, 0, 2], draft[0, 0, 2] = p, q
    tokens = torch.tensor([[2]], dtype=torch.int32)
    n, out = ds4.verify_drafts(target.cuda(), draft.cuda(), tokens.cuda(), torch.tensor([[u]]).cuda(),
                               torch.tensor([1 - 2.0 ** -24]).cuda())
    assert n.tolist() == [int(accepted)]
    assert out.tolist() == [[2, 4] if accepted else [4, -1]]
