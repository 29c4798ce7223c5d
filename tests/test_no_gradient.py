"""Calls without a gradient refuse tensors that require one while autograd records, where their result would have none, or
one of values that have been moved (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def om():
    import ordered_merge_gb300

    return ordered_merge_gb300


def _calls(om):
    """Each call as a function of the tensor that may require a gradient, and that tensor."""
    half = lambda *s: torch.randn(*s).bfloat16()  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x, w, up, down = half(4, 16), torch.randn(4, 2), half(5, 8, 16), half(5, 16, 8)
    yield lambda t: om.expert_mlp(t, i32(4, 2), w, up, down), x
    yield lambda t: om.expert_mlp(x, i32(4, 2), t, up, down), w
    yield lambda t: om.expert_mlp(x, i32(4, 2), w, t, down), up
    yield lambda t: om.expert_mlp(x, i32(4, 2), w, up, t), down
    yield lambda t: om.expert_mlp(x, i32(4, 2), w, up, down, gate=t), half(5, 8, 16)
    yield lambda t: om.expert_mlp(x, i32(4, 2), w, up, down, out=t), half(4, 16)
    state = torch.randn(2, 3, 1, 4)
    yield lambda t: om.beam_gather(i32(2, 3), (state, t)), torch.randn(2, 3, 1, 4)
    yield lambda t: om.beam_gather(i32(2, 3), (t,), out=(state,)), torch.randn(2, 3, 1, 4)
    yield lambda t: om.beam_gather(i32(2, 3), (state,), out=(t,)), torch.randn(2, 3, 1, 4)
    ids = torch.tensor([1, 4])
    yield lambda t: om.embed_lookup(ids, torch.randn(6, 8), out=t), torch.randn(2, 8)
    yield lambda t: om.beam_select(torch.randn(2, 3, 9), 2, out_scores=t), torch.randn(2, 2)
    yield lambda t: om.embed_lookup_backward(t, ids, 6), torch.randn(2, 8)
    yield lambda t: om.embed_lookup_backward(torch.randn(2, 8), ids, 6, accumulate=True, grad_table=t), torch.randn(6, 8)


def test_refused_while_autograd_records(om):
    for call, t in _calls(om):
        with pytest.raises(ValueError, match="has no gradient"):
            call(t.clone().requires_grad_())
        with pytest.raises(ValueError, match="has no gradient"):
            call(t.clone().requires_grad_() * 1)


@pytest.mark.gpu
def test_taken_without_a_record(gpu):
    gen = torch.Generator(device="cuda").manual_seed(0)
    half = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, up, down = half(4, 16), torch.nn.Parameter(half(5, 8, 16)), torch.nn.Parameter(half(5, 16, 8))
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.ones(4, 2, device="cuda")
    want = gpu.expert_mlp(x, ids, w, up.detach(), down.detach())
    with pytest.raises(ValueError, match="has no gradient"):
        gpu.expert_mlp(x, ids, w, up, down)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(gpu.expert_mlp(x, ids, w, up, down), want)
            state = torch.nn.Parameter(torch.randn(1, 2, 1, 3, device="cuda"))
            moved = state[:, [1, 1]].clone()
            gpu.beam_gather(torch.ones(1, 2, dtype=torch.int32, device="cuda"), (state,))
            assert torch.equal(state, moved)
    # where autograd asks for a gradient of the gradient, the rows' own node refuses
    table = torch.randn(6, 8, device="cuda", requires_grad=True)
    rows = gpu.embed_lookup(torch.tensor([1, 4], device="cuda"), table)
    grad, = torch.autograd.grad((rows * rows).sum(), table, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()
