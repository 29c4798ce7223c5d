"""om_expert_mlp with infinite weights of the second product: an infinity of its sign where the activation is a number other
than zero, as the formula has it, although an activation goes there as two values, of which one may be zero or negative."""
import pytest
import torch

from test_gpu_experts import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("hidden,inner", [(64, 48), (63, 47), (1032, 1100)])
def test_infinite_weights_of_the_second_product(gpu, dtype, gated, hidden, inner):
    case = _case(5, 2, 4, hidden, inner, dtype, gated)
    case["ids"] = torch.tensor([[0, 1], [1, 2], [2, 3], [3, 3], [0, 3]], dtype=torch.int32, device="cuda")
    want = gpu.expert_mlp(**case)
    up, e, k = case["up"], 2, inner - 3
    # its activation is a whole number for one token, so that its rounding leaves nothing, and of any bits for another
    case["x"][2], up[e, k] = 0, 0
    case["x"][2, 0], up[e, k, 0] = 1, 2
    if gated:
        case["gate"][e, k] = 0
        case["gate"][e, k, 0] = 3
    case["x"][1, 0] = 0.7310
    plain = gpu.expert_mlp(**case, act="relu")
    assert plain.isfinite().all()
    case["down"][e, 3, k], case["down"][e, 7, k] = float("inf"), -float("inf")
    got = gpu.expert_mlp(**case, act="relu")
    for t in (1, 2):  # the tokens of expert 2
        assert got[t, 3] == float("inf") and got[t, 7] == -float("inf")
    got[1:3, 3], got[1:3, 7] = plain[1:3, 3], plain[1:3, 7]
    assert torch.equal(got, plain)
    assert torch.equal(gpu.expert_mlp(**case)[[0, 3, 4]], want[[0, 3, 4]])
