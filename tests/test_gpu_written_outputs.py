"""Tensors handed to the library as outputs, or changed in place, are known to autograd as changed: a backward pass that
saved what stood there before refuses, instead of giving the gradient of other values."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(om):
    """(what is called, the tensors that it writes) for every output that can be handed in."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    new = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    logits, out = rand(2, 3, 50), [new(2, 3, dtype=torch.float32), new(2, 3), new(2, 3)]
    yield lambda: om.beam_select(logits, 3, out_scores=out[0], parents=out[1], tokens=out[2]), out
    parents, states, into = new(2, 3), [rand(2, 3, 2, 5, 4), rand(2, 3, 2, 5)], [rand(2, 3, 2, 5, 4), rand(2, 3, 2, 5)]
    yield lambda: om.beam_gather(parents, states), states
    yield lambda: om.beam_gather(parents, states, out=into), into
    ids, table, rows, grads = torch.tensor([1, 4, 4], device="cuda"), rand(6, 8), rand(3, 8), rand(6, 8)
    yield lambda: om.embed_lookup(ids, table, out=rows), [rows]
    yield lambda: om.embed_lookup_backward(rand(3, 8), ids, 6, grad_table=grads), [grads]
    yield lambda: om.embed_lookup_backward(rand(3, 8), ids, 6, accumulate=True, grad_table=grads), [grads]
    half = lambda *s: rand(*s).bfloat16()  # noqa: E731
    x, up, down, y = half(4, 16), half(5, 8, 16), half(5, 16, 8), half(4, 16)
    yield lambda: om.expert_mlp(x, new(4, 2), rand(4, 2), up, down, out=y), [y]
    scores, e, w, g = rand(4, 8), new(4, 2), new(4, 2, dtype=torch.float32), rand(4, 8)
    yield lambda: om.route_topk(scores, 2, ids=e, weights=w), [e, w]
    yield lambda: om.route_topk(scores.clone().requires_grad_(), 2, ids=e, weights=w.detach()), [e, w]
    yield lambda: om.route_topk_backward(scores, e, rand(4, 2), grad_logits=g), [g]
    groups = [new(9), new(8), new(8)]
    yield lambda: om.group_by_id(e.flatten(), 8, offsets=groups[0], order=groups[1], place=groups[2]), groups
    weights, total = rand(2, 4, 3, 20).softmax(3), rand(2, 2, 20)
    yield lambda: om.accumulate_weights(weights, total, out=total), [total]
    keep = [new(2, 2, 5), new(2)]
    yield lambda: om.evict_select(total, 5, keep=keep[0], kept=keep[1]), keep
    cache = rand(2, 2, 20, 4)
    yield lambda: om.evict_gather(keep[0], (cache,), out=(cache[:, :, :5],)), [cache]


def test_versions_rise(gpu):
    for call, written in _calls(gpu):
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before))


def test_inputs_keep_their_versions(gpu):
    logits, ids, table = torch.randn(2, 3, 50, device="cuda"), torch.tensor([1, 4], device="cuda"), torch.randn(6, 8, device="cuda")
    scores = torch.zeros(2, 3, device="cuda")
    before = [t._version for t in (logits, scores, ids, table)]
    parents = gpu.beam_select(logits, 3, scores)[1]
    version = parents._version
    gpu.beam_gather(parents, (torch.zeros(2, 3, 1, 4, device="cuda"),))
    gpu.embed_lookup(ids, table)
    assert before == [t._version for t in (logits, scores, ids, table)] and parents._version == version


def test_saved_states_that_move_in_place(gpu):
    parents = torch.tensor([[1, 1]], dtype=torch.int32, device="cuda")
    states, w = torch.randn(1, 2, 1, 3, 4, device="cuda"), torch.ones(4, device="cuda", requires_grad=True)
    loss = (states * w).sum()  # saves the states for the gradient of w
    gpu.beam_gather(parents, (states,))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_saved_ids_that_the_next_step_writes_over(gpu):
    """A buffer of tokens that every step of a search fills: an earlier step's rows still need what it held."""
    table = torch.randn(50, 8, device="cuda", requires_grad=True)
    out = [torch.zeros(2, 3, device="cuda"), *(torch.zeros(2, 3, dtype=torch.int32, device="cuda") for _ in range(2))]
    select = lambda: gpu.beam_select(torch.randn(2, 3, 50, device="cuda"), 3, out_scores=out[0], parents=out[1], tokens=out[2])  # noqa: E731
    loss = gpu.embed_lookup(select()[2], table).sum()
    loss.backward()
    loss = gpu.embed_lookup(select()[2], table).sum()
    select()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_made_under_inference_mode(gpu):
    """Such tensors have no version to raise; the calls write them as others."""
    with torch.inference_mode():
        table, out = torch.randn(6, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
        ids = torch.tensor([3, 0], device="cuda")
        gpu.embed_lookup(ids, table, out=out)
        assert torch.equal(out, table[ids])
        states = torch.randn(1, 2, 1, 3, device="cuda")
        want = states[:, [1, 1]].clone()
        gpu.beam_gather(torch.tensor([[1, 1]], dtype=torch.int32, device="cuda"), (states,))
        assert torch.equal(states, want)
    gpu.embed_lookup(ids.clone(), table.clone(), out=out)
