"""om_expert_mlp's activations far out, where they are small differences of great values, against 64 bits."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu


def _layer(dtype, values, gated, rows):
    """A layer whose output r is 2^14 * 2^k * act(values[r]), each sum of one term; values are of the type."""
    n = len(values)
    up = torch.zeros(1, rows, rows, device="cuda", dtype=dtype)
    gate = up.clone()
    (gate if gated else up)[0, :n, 0] = values
    if gated:
        up[0, :n, 0] = 1
    down = torch.zeros(1, rows, rows, device="cuda", dtype=dtype)
    at = torch.arange(n, device="cuda")
    down[0, at, at] = 2.0 ** 14
    x = torch.zeros(1, rows, device="cuda", dtype=dtype)
    x[0, 0] = 1
    return dict(x=x, ids=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), weights=torch.ones(1, 1, device="cuda"), up=up,
                down=down, gate=gate if gated else None)


def _act(act, u):
    u = u.double()
    if act == "gelu":
        return 0.5 * u * torch.special.erfc(-u * 0.5 ** 0.5)
    return u / (1 + torch.exp(-u)) if act == "silu" else u.clamp(min=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [64, 63])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_activations_far_out(gpu, dtype, gated, rows, act):
    """gelu's argument of erfc is within 1.5 * 2^-24 of itself, which the function's slope makes 2 y^2 + 1 = 26 times as
    much at y = 5 / sqrt 2; erfc itself is within 4 units, a product rounds once: 2^-18 in all.  silu's exponential is
    within 2 units, its argument exact.  The pair of values holds the rest to 2^-16, or to 2^-36 in f16, which is 2^-16 of
    gelu(-5)."""
    values = torch.cat([torch.linspace(-5, -0.0625, 40), torch.linspace(0.0625, 3.5, 20)]).cuda().to(dtype)
    got = gpu.expert_mlp(**_layer(dtype, values, gated, rows), act=act)[0, :60].double()
    want = 2.0 ** 14 * _act(act, values)
    assert torch.all((got - want).abs() <= (ref.HALF[dtype] + 2.0 ** -15 + 2.0 ** -18) * want.abs() + 2.0 ** -25)
