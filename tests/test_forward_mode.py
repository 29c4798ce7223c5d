"""Tensors with a forward-mode tangent are refused: the calls would drop it without a word (no GPU needed)."""
import pytest
import torch
from torch.autograd import forward_ad


@pytest.fixture(scope="module")
def om():
    import ordered_merge_gb300

    return ordered_merge_gb300


def _calls(om):
    """Each call as a function of the tensor that may carry a tangent, and that tensor."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    half = lambda *s: torch.randn(*s).bfloat16()  # noqa: E731
    ids, up, down = torch.tensor([1, 4]), half(5, 8, 16), half(5, 16, 8)
    yield lambda t: om.embed_lookup(ids, t), torch.randn(6, 8)
    yield lambda t: om.embed_lookup_backward(t, ids, 6), torch.randn(2, 8)
    yield lambda t: om.beam_select(t, 2), torch.randn(2, 3, 9)
    yield lambda t: om.beam_select(torch.randn(2, 3, 9), 2, t), torch.randn(2, 3)
    yield lambda t: om.beam_gather(i32(2, 3), (torch.zeros(2, 3, 1, 4), t)), torch.randn(2, 3, 1, 4)
    yield lambda t: om.beam_gather(i32(2, 3), (t,), out=(torch.zeros(2, 3, 1, 4),)), torch.randn(2, 3, 1, 4)
    yield lambda t: om.expert_mlp(t, i32(4, 2), torch.randn(4, 2), up, down), half(4, 16)
    yield lambda t: om.expert_mlp(half(4, 16), i32(4, 2), torch.randn(4, 2), up, t), down
    yield lambda t: om.expert_mlp(half(4, 16), i32(4, 2), t, up, down), torch.randn(4, 2)
    yield lambda t: om.route_topk(t, 2), torch.randn(4, 8)
    yield lambda t: om.route_topk_backward(torch.randn(4, 8), i32(4, 2), t), torch.randn(4, 2)
    yield lambda t: om.accumulate_weights(t, kv_heads=2), torch.randn(2, 4, 3, 20)
    yield lambda t: om.evict_select(t, 5), torch.randn(2, 2, 20)
    yield lambda t: om.evict_gather(i32(2, 2, 5), (t,)), torch.randn(2, 2, 20, 4)


def test_tangents_are_refused(om):
    for call, t in _calls(om):
        with forward_ad.dual_level():
            with pytest.raises(ValueError, match="tangent"):
                call(forward_ad.make_dual(t, torch.ones_like(t)))


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu(gpu):
    table = torch.randn(6, 8, device="cuda")
    ids = torch.tensor([1, 4], device="cuda")
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(table, torch.ones_like(table))
        with pytest.raises(ValueError, match="table carries a forward-mode tangent"):
            gpu.embed_lookup(ids, dual)
        # where a gradient is recorded, autograd itself refuses it
        leaf = table.clone().requires_grad_()
        with pytest.raises((ValueError, NotImplementedError)):
            gpu.embed_lookup(ids, forward_ad.make_dual(leaf, torch.ones_like(leaf)))
        # tensors without one are as outside, and a primal alone is taken
        assert torch.equal(gpu.embed_lookup(ids, table), table[ids])
        assert torch.equal(gpu.embed_lookup(ids, forward_ad.unpack_dual(dual).primal), table[ids])
