"""om_route_topk in a training loop: weights that carry their gradient to the logits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

OPTIONS = dict(score="sigmoid", groups=4, group_picks=2, group_best=2, renorm=True, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("options", [dict(), dict(renorm=True), OPTIONS], ids=["softmax", "renorm", "groups"])
def test_weights_carry_the_gradient(gpu, dtype, options):
    x = torch.randn(70, 64, device="cuda").to(dtype)
    bias = torch.randn(64, device="cuda") * 0.01
    pull = torch.randn(70, 6, device="cuda")
    ids, w = gpu.route_topk(x, 6, bias=bias, **options)
    assert not w.requires_grad
    leaf = x.clone().requires_grad_()
    ids2, w2 = gpu.route_topk(leaf * 1, 6, bias=bias, **options)
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and w2.requires_grad and not ids2.requires_grad
    (w2 * pull).sum().backward()
    back = {k: v for k, v in options.items() if k in ("score", "renorm", "scale")}
    assert torch.equal(leaf.grad, gpu.route_topk_backward(x, ids, pull, **back))
    with torch.no_grad():
        assert not gpu.route_topk(leaf, 6, **options)[1].requires_grad


def test_gradients_that_are_not_contiguous(gpu):
    leaf = torch.randn(9, 16, device="cuda", requires_grad=True)
    ids, w = gpu.route_topk(leaf, 3)
    w.sum().backward()  # a gradient of stride 0
    assert torch.equal(leaf.grad, gpu.route_topk_backward(leaf.detach(), ids, torch.ones_like(w)))


def test_given_outputs(gpu):
    """Outputs that are handed in are filled, and the weights among them carry the gradient."""
    leaf = torch.randn(9, 16, device="cuda", requires_grad=True)
    ids, w = torch.empty(9, 3, dtype=torch.int32, device="cuda"), torch.empty(9, 3, device="cuda")
    got = gpu.route_topk(leaf, 3, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w and w.requires_grad
    (w * w).sum().backward()
    plain = gpu.route_topk(leaf.detach(), 3)
    assert torch.equal(ids, plain[0])
    assert torch.equal(leaf.grad, gpu.route_topk_backward(leaf.detach(), ids, 2 * plain[1]))


def test_rows_that_share_memory(gpu):
    """One row of logits for every token: its gradient is the sum."""
    row = torch.randn(32, device="cuda", requires_grad=True)
    ids, w = gpu.route_topk(row.expand(20, 32), 4)
    pull = torch.randn(20, 4, device="cuda")
    (w * pull).sum().backward()
    each = gpu.route_topk_backward(row.detach().expand(20, 32), ids, pull)
    assert torch.allclose(row.grad, each.sum(0), rtol=1e-5, atol=1e-6)


def test_outputs_used_again_at_every_step(gpu):
    """Buffers that a training loop keeps: each step's backward pass is its own."""
    ids, room = torch.empty(9, 3, dtype=torch.int32, device="cuda"), torch.empty(20, 3, device="cuda")
    for buffer in (torch.empty(9, 3, device="cuda"), room[4:13]):
        for _ in range(3):
            leaf = torch.randn(9, 16, device="cuda", requires_grad=True)
            _, w = gpu.route_topk(leaf, 3, ids=ids, weights=buffer)
            (w * w).sum().backward()
            plain = gpu.route_topk(leaf.detach(), 3)
            assert torch.equal(leaf.grad, gpu.route_topk_backward(leaf.detach(), plain[0], 2 * plain[1]))
        late = torch.randn(9, 16, device="cuda", requires_grad=True)
        _, w = gpu.route_topk(late, 3, ids=ids, weights=buffer)
        loss = (w * w).sum()
        gpu.route_topk(torch.randn(9, 16, device="cuda", requires_grad=True), 3, ids=ids, weights=buffer)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()  # its weights have been written over


def test_second_derivatives_are_refused(gpu):
    leaf = torch.randn(9, 16, device="cuda", requires_grad=True)
    _, w = gpu.route_topk(leaf, 3)
    grad, = torch.autograd.grad((w * w).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()
