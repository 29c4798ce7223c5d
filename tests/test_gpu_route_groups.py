"""Groups of om_route_topk without an expert, beside groups whose sum leaves the range of 32 bits."""
import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [3, 2600])
@pytest.mark.parametrize("experts,groups,picks,k", [(32, 4, 2, 12), (32, 8, 2, 8), (64, 8, 3, 8), (48, 3, 2, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_empty_group_takes_no_place(gpu, tokens, experts, groups, picks, k, score):
    """A bias of the type's lowest value masks all but the first group, whose logits are -inf: the sums of two are
    all -inf, and still the first groups that have experts are picked."""
    size = experts // groups
    x = torch.zeros(tokens, experts)
    x[:, :size] = -float("inf")
    bias = torch.full((experts,), torch.finfo(torch.float32).min)
    ids, _ = gpu.route_topk(x.cuda(), k, score=score, bias=bias.cuda(), groups=groups, group_picks=picks, group_best=2)
    want, _ = ref.route(f64(x[:2]), k, score, f64(bias), groups, picks, 2)
    assert (want >= size).sum() >= min(k, picks * size) * 2
    assert np.array_equal(ids.cpu().numpy()[:2], want) and (ids == ids[0]).all()
