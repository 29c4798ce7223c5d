"""The order of om_route_topk's choices where scores leave the normal range, and the same from all its kernels.

No bias, several groups, two greatest scores to a group: the choice is by the scores in 32 bits.
"""
import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import f64

pytestmark = pytest.mark.gpu

FEW, MANY = 3, 2600  # tokens that get 32 and 8 lanes each


@pytest.mark.parametrize("tokens", [FEW, MANY])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_below_the_normal_range_keep_their_order(gpu, tokens, dtype):
    """Sigmoid scores from e^-88 to e^-96, a quarter (bf16: a half, at least 64 %) apart: subnormal, but distinct."""
    step = 0.25 if dtype == torch.float32 else 0.5
    gen = torch.Generator().manual_seed(7)
    x = torch.stack([-80.0 - 8 - step * torch.randperm(32 if step == 0.25 else 16, generator=gen) for _ in range(tokens)])
    x = torch.cat([x, torch.full_like(x, -float("inf"))], 1) if step == 0.5 else x
    x = x.to(dtype)
    ids, _ = gpu.route_topk(x.cuda(), 8, score="sigmoid", groups=2, group_picks=2, group_best=2, renorm=True)
    rows = list(range(0, tokens, max(1, tokens // 40)))
    want, _ = ref.route(f64(x[rows]), 8, "sigmoid", groups=2, group_picks=2, group_best=2, renorm=True)
    assert np.array_equal(ids.cpu().numpy()[rows], want)


@pytest.mark.parametrize("tokens", [FEW, MANY])
@pytest.mark.parametrize("k", [8, 12])
def test_kernels_choose_alike(gpu, tokens, k):
    """All groups open: two groups (lists) and three (a warp a token) rank the same experts by the same scores."""
    gen = torch.Generator().manual_seed(k)
    rows = {
        "spread": torch.randn(tokens, 96, generator=gen) * 8,
        "saturated": 15 + torch.randint(0, 64, (tokens, 96), generator=gen) / 8,
        "low": -86 - torch.randint(0, 120, (tokens, 96), generator=gen) / 8,
        "close": 1 + torch.randint(0, 4000, (tokens, 96), generator=gen) * 2.0 ** -22,
    }
    for name, x in rows.items():
        a, _ = gpu.route_topk(x.cuda(), k, score="sigmoid", groups=2, group_picks=2, group_best=2)
        b, _ = gpu.route_topk(x.cuda(), k, score="sigmoid", groups=3, group_picks=3, group_best=2)
        assert torch.equal(a, b), name
