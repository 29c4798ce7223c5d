"""om_expert_mlp on layers of more columns than one block of the kernel takes at once, and on rows that no vector fits,
against the definition in 64 bits."""
import pytest
import torch

from test_gpu_experts import _case, _check

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("hidden,inner", [(1024, 1024), (1032, 1016), (1016, 1032), (2048, 1056), (2056, 2040), (72, 2600), (4104, 40)])
def test_several_blocks_of_columns(gpu, dtype, gated, hidden, inner):
    for tokens, picks, experts in ((1, 2, 3), (10, 2, 4), (24, 1, 2)):
        _check(gpu, **_case(tokens, picks, experts, hidden, inner, dtype, gated))


@pytest.mark.parametrize("dtype", TYPES)
def test_every_column_and_row_counts(gpu, dtype):
    """Sums of small whole numbers, exact in 32 bits and in the type: nothing may be lost, or counted twice."""
    hidden, inner, experts = 2072, 1304, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(9, hidden, device="cuda")
    x.scatter_(1, torch.randint(0, hidden, (9, 40), generator=gen, device="cuda"), 1.0)
    up = (torch.rand(experts, inner, hidden, generator=gen, device="cuda") < 0.02).float()
    down = (torch.rand(experts, hidden, inner, generator=gen, device="cuda") < 0.02).float()
    ids = torch.randint(0, experts, (9, 2), generator=gen, device="cuda", dtype=torch.int32)
    weights = torch.ones(9, 2, device="cuda")
    got = gpu.expert_mlp(x.to(dtype), ids, weights, up.to(dtype), down.to(dtype), act="relu")
    want = torch.zeros(9, hidden, dtype=torch.float64, device="cuda")
    for t in range(9):
        for e in ids[t].tolist():
            want[t] += down[e].double() @ (up[e].double() @ x[t].double())
    assert float(want.max()) <= 128  # whole numbers that bf16 holds
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("hidden,inner", [(2001, 1399), (1025, 7), (7, 1025), (1031, 1024)])
def test_odd_rows_of_many_columns(gpu, dtype, gated, hidden, inner):
    for tokens, picks, experts in ((2, 2, 3), (20, 1, 1), (37, 2, 2)):
        _check(gpu, **_case(tokens, picks, experts, hidden, inner, dtype, gated))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["x", "up", "gate", "down"])
def test_rows_at_any_address(gpu, dtype, which):
    """One of the inputs at an address, or with a stride, that no vector allows."""
    for shift in range(1, 8):
        case = _case(6, 2, 4, 80, 48, dtype, True, seed=shift)
        shape = case[which].shape
        apart = (*shape[:-1], shape[-1] + (shift if shift % 2 else 0))
        room = torch.full((torch.Size(apart).numel() + 8,), float("nan"), device="cuda", dtype=dtype)
        view = room[shift:shift + torch.Size(apart).numel()].view(apart)[..., :shape[-1]]
        view.copy_(case[which])
        case[which] = view
        _check(gpu, **case)


@pytest.mark.parametrize("dtype", TYPES)
def test_gelu_and_silu_of_many_columns(gpu, dtype):
    for act in ("gelu", "silu"):
        for gated in (False, True):
            _check(gpu, act, **_case(5, 2, 3, 1064, 1208, dtype, gated))
            _check(gpu, act, **_case(5, 2, 3, 1063, 1207, dtype, gated))
