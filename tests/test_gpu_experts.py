"""om_expert_mlp against its definition in 64 bits."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu


def _case(tokens, picks, experts, hidden, inner, dtype, gated, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + tokens * 1000 + hidden)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ids = torch.rand(tokens, experts, generator=gen, device="cuda").argsort(1)[:, :picks].int().contiguous()
    w = rand(tokens, ids.shape[1]).softmax(1)
    mat = lambda r, c: (rand(experts, r, c) * c ** -0.5).to(dtype)  # noqa: E731
    return dict(x=rand(tokens, hidden).to(dtype), ids=ids, weights=w, up=mat(inner, hidden), down=mat(hidden, inner),
                gate=mat(inner, hidden) if gated else None)


def _check(om, act="silu", out=None, **case):
    ref.DT[0] = case["x"].dtype
    got = om.expert_mlp(**case, act=act, out=out)
    want, error = ref.expert_mlp(**case, act=act)
    bound = error + ref.HALF[got.dtype] * (want.abs() + error) + 2.0 ** -25
    assert torch.all((got.double() - want).abs() <= bound)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("hidden,inner", [(8, 8), (64, 32), (128, 104), (520, 264), (33, 17), (1, 1), (100, 250), (264, 31)])
def test_sizes(gpu, dtype, gated, hidden, inner):
    for tokens, picks, experts in ((1, 1, 1), (1, 4, 9), (3, 2, 40), (9, 3, 5), (21, 1, 2)):
        _check(gpu, **_case(tokens, picks, experts, hidden, inner, dtype, gated))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(gpu, act, gated):
    case = _case(5, 2, 6, 96, 64, torch.bfloat16, gated)
    case["x"] *= 4
    _check(gpu, act, **case)


@pytest.mark.parametrize("tokens", [1, 2, 8, 16, 17, 33, 64])
@pytest.mark.parametrize("experts,picks", [(1, 1), (2, 2), (4, 1), (64, 8), (300, 2), (1024, 3)])
def test_tokens_and_experts(gpu, tokens, experts, picks):
    """From one expert that has every token to more experts than slots."""
    _check(gpu, **_case(tokens, picks, experts, 72, 40, torch.bfloat16, True))


def test_all_tokens_ask_for_one_of_many(gpu):
    """One expert has all the tokens, several batches of them, among many experts and with more slots than experts."""
    for experts, picks in ((300, 1), (7, 3)):
        case = _case(64, picks, experts, 64, 48, torch.float16, True)
        case["ids"][:] = experts - 1 if picks == 1 else torch.tensor([4, 0, 2], device="cuda", dtype=torch.int32)
        _check(gpu, **case)


def test_empty_slots(gpu):
    case = _case(6, 3, 8, 64, 32, torch.bfloat16, True)
    case["ids"][0, 1], case["ids"][1], case["ids"][2, 0], case["ids"][3, 2] = -1, -1, 8, -(1 << 31)
    case["weights"][0, 1] = float("nan")  # an empty slot counts for nothing
    got = gpu.expert_mlp(**case)
    assert not got[1].any() and not got.isnan().any()
    case["weights"][0, 1] = 0.0
    assert torch.equal(_check(gpu, **case), got)
    case["ids"][:] = -1
    assert not gpu.expert_mlp(**case).any()


def test_the_same_expert_twice(gpu):
    case = _case(4, 4, 5, 64, 32, torch.float16, True)
    case["ids"][:] = torch.tensor([[1, 1, 1, 1], [0, 2, 2, 0], [3, 3, 4, 4], [2, 1, 0, 2]], dtype=torch.int32, device="cuda")
    first = _check(gpu, **case)
    for _ in range(5):
        assert torch.equal(gpu.expert_mlp(**case), first)


def test_strides_and_one_array_for_gate_and_up(gpu):
    case = _case(7, 2, 6, 80, 48, torch.bfloat16, True)
    want = gpu.expert_mlp(**case)
    both = torch.cat([case["gate"], case["up"]], 1)
    got = gpu.expert_mlp(case["x"], case["ids"], case["weights"], both[:, 48:], case["down"], gate=both[:, :48])
    assert torch.equal(got, want)
    wide = torch.zeros(7, 96, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:88] = case["x"]
    out = torch.full((7, 100), 3.0, dtype=torch.bfloat16, device="cuda")
    gpu.expert_mlp(wide[:, 8:88], case["ids"], case["weights"], case["up"], case["down"], gate=case["gate"], out=out[:, 5:85])
    assert torch.equal(out[:, 5:85], want) and torch.all(out[:, :5] == 3) and torch.all(out[:, 85:] == 3)
    for shift in range(1, 8):  # rows at addresses that no vector allows
        odd = torch.zeros(6 * 80 * 48 + 8, dtype=torch.bfloat16, device="cuda")[shift:shift + 6 * 80 * 48].view(6, 80, 48)
        odd.copy_(case["down"])
        got = gpu.expert_mlp(case["x"], case["ids"], case["weights"], case["up"], odd, gate=case["gate"])
        assert torch.all((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 1e-3 * want.abs().max())


def test_values_that_are_not_finite(gpu):
    case = _case(4, 2, 5, 64, 32, torch.bfloat16, False)
    case["ids"] = torch.tensor([[0, 1], [2, 3], [2, 4], [3, 4]], dtype=torch.int32, device="cuda")
    want = gpu.expert_mlp(**case)
    case["x"][0, 3] = float("nan")
    case["up"][1, 5, 6] = float("inf")
    got = gpu.expert_mlp(**case)
    assert got[0].isnan().all() and torch.equal(got[1:], want[1:])  # other tokens are as before
    case["x"][1, 0] = float("inf")
    got = gpu.expert_mlp(**case)
    assert not got[1].isfinite().any() and torch.equal(got[2:], want[2:])


def test_streams_repeats_and_weights_past_32_bits(gpu):
    case = _case(16, 4, 12, 128, 64, torch.bfloat16, True)
    want = gpu.expert_mlp(**case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = gpu.expert_mlp(**case, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    experts, hidden, inner = 600, 2048, 2048  # 5 GB to each matrix
    up = torch.zeros(experts, inner, hidden, dtype=torch.bfloat16, device="cuda")
    down = torch.zeros(experts, hidden, inner, dtype=torch.bfloat16, device="cuda")
    up[-1, 7, 5], up[1, 7, 5], down[-1, 9, 7], down[1, 9, 7] = 2.0, 3.0, 4.0, 5.0
    x = torch.zeros(2, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, 5] = 1.0
    ids = torch.tensor([[experts - 1], [1]], dtype=torch.int32, device="cuda")
    got = gpu.expert_mlp(x, ids, torch.ones(2, 1, device="cuda"), up, down, act="relu")
    assert got[0, 9] == 8 and got[1, 9] == 15 and got.count_nonzero() == 2


def test_after_route_topk(gpu):
    """Ids and weights as the router gives them, masked experts among them."""
    case = _case(12, 4, 32, 64, 40, torch.bfloat16, True)
    logits = torch.randn(12, 32, device="cuda")
    logits[3, 2:] = -float("inf")
    logits[4] = -float("inf")
    case["ids"], case["weights"] = gpu.route_topk(logits, 4, renorm=True)
    got = _check(gpu, **case)
    assert not got[4].any()
