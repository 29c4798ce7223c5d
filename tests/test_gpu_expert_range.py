"""om_expert_mlp's activations between its two products, down to small ones.

The layers here make each activation an exact product of two values of the type (22 or 16 bits), and each output the
difference of such an activation and its own rounding, times powers of two: what the kernels keep beyond one value."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def _residuals(dtype, rows, power, experts=2, tokens=3, seed=0):
    """(case, want, |h|): out[t, r] = weight * 2^10 * (h - rounded h) with h of about 2^power."""
    gen = torch.Generator(device="cuda").manual_seed(seed + rows - power)
    rand = lambda *s: 1 + torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    left = power // 2
    g, u = (rand(experts, rows) * 2.0 ** left).to(dtype), (rand(experts, rows) * 2.0 ** (power - left)).to(dtype)
    h = g.double() * u.double()
    rounded = h.to(dtype)  # h is exact in 32 bits, so this is one rounding
    gate = torch.zeros(experts, 2 * rows, rows, device="cuda", dtype=dtype)
    up, down = gate.clone(), torch.zeros(experts, rows, 2 * rows, device="cuda", dtype=dtype)
    gate[:, :rows, 0], up[:, :rows, 0] = g, u
    gate[:, rows:, 0], up[:, rows:, 0] = 1, rounded
    at = torch.arange(rows, device="cuda")
    down[:, at, at], down[:, at, at + rows] = 2.0 ** 10, -2.0 ** 10
    x = torch.zeros(tokens, rows, device="cuda", dtype=dtype)
    x[:, 0] = 1
    ids = (torch.arange(tokens, device="cuda", dtype=torch.int32) % experts)[:, None].contiguous()
    # what is left of h is at most half a step of the type: outputs of about 1
    weight = 2.0 ** -10 / max(2.0 ** power * ref.HALF[dtype], 2.0 ** -25 if dtype == torch.float16 else 0.0)
    case = dict(x=x, ids=ids, weights=torch.full((tokens, 1), weight, device="cuda"), up=up, down=down, gate=gate)
    e = ids[:, 0].long()
    return case, weight * 2.0 ** 10 * (h - rounded.double())[e], weight * 2.0 ** 10 * h[e]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("power", [0, -2, -4, -6, -8, -10, -12, -14, -16, -18, -20])
@pytest.mark.parametrize("rows", [64, 40, 63], ids=["aligned", "short", "odd"])
def test_small_activations_keep_their_bits(gpu, dtype, power, rows):
    """The pair of values holds h to half a step of half a step: 2^-16 of it in bf16, 2^-22 in f16, and no less than the
    half of 2^-24 / 2^11 that f16 has there.  The rounded h cancels exactly, so nothing else is added but the output's
    rounding."""
    case, want, h = _residuals(dtype, rows, power)
    got = gpu.expert_mlp(**case, act="relu").double()
    unit = h / torch.where(h != 0, h, 1.0)  # of one activation's scale
    assert torch.all(unit == 1)
    scale = float(case["weights"][0, 0]) * 2.0 ** 10
    least = scale * 2.0 ** -36 if dtype == torch.float16 else 0.0
    bound = ref.HALF[dtype] ** 2 * h + least + (ref.HALF[dtype] + 2 * ref.E32) * want.abs() + 2.0 ** -25
    assert torch.all((got - want).abs() <= bound)


@pytest.mark.parametrize("tokens,experts", [(1, 4), (20, 2), (64, 3)])
def test_small_activations_of_many_tokens(gpu, tokens, experts):
    for rows in (72, 71):
        case, want, h = _residuals(torch.float16, rows, -9, experts, tokens)
        got = gpu.expert_mlp(**case, act="relu").double()
        bound = 2.0 ** -22 * h + (2.0 ** -11 + 2 * ref.E32) * want.abs() + 2.0 ** -25
        assert torch.all((got - want).abs() <= bound)


def test_the_ends_of_f16(gpu):
    """The greatest finite activation keeps what its rounding left; beyond it the first value is infinite, and the
    second adds nothing to it (no NaN)."""
    for rows in (16, 15):
        case, _, _ = _residuals(torch.float16, rows, 0, 1, 1)
        case["weights"][:] = 2.0 ** -17
        for g, u in ((255.875, 255.875), (255.0, 256.75), (2.0, 32752.0), (-1.0, 5.0)):
            case["gate"][:, :rows, 0], case["up"][:, :rows, 0] = g, u
            case["up"][:, rows:, 0] = 1.0
            got = gpu.expert_mlp(**case, act="relu").double()
            want = (max(g, 0.0) * u - 1.0) * 2.0 ** -7
            assert torch.all((got - want).abs() <= 2.0 ** -22 * abs(want) + (2.0 ** -11 + 2 * ref.E32) * abs(want) + 2.0 ** -25)
        case["gate"][:, 0, 0], case["up"][:, 0, 0] = 256.0, 256.0
        assert torch.all(gpu.expert_mlp(**case, act="relu")[:, 0] == float("inf"))
