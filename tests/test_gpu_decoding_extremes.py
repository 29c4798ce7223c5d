"""The calls of a decoding step past 32-bit offsets, from several host threads, and captured on every way that they take."""
import threading

import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("width", [2200, 2201])
def test_gradient_past_32_bits(gpu, width):
    """More than 4 GB of the rows' gradient, and of the table's: a permutation moves every row whole."""
    n = 1 << 20
    order = torch.randperm(n, generator=_gen(1), device="cuda")
    grad = torch.randint(-64, 64, (n, width), generator=_gen(2), device="cuda", dtype=torch.int8).half()
    got = gpu.embed_lookup_backward(grad, order, n)
    for rows in (slice(0, 1000), slice(n // 2, n // 2 + 1000), slice(n - 1000, n)):
        assert torch.equal(got[order[rows]], grad[rows])
    few = torch.tensor([n - 1, 5, n - 1], device="cuda")
    gpu.embed_lookup_backward(grad[:3].contiguous(), few, n, accumulate=True, grad_table=got)
    want = grad[order.argsort()[n - 1]].float() + grad[0].float() + grad[2].float()
    assert torch.equal(got[n - 1].float(), want)  # small whole numbers
    got.fill_(7.0)
    gpu.embed_lookup_backward(grad[:3].contiguous(), few, n, grad_table=got)
    assert torch.equal(got[5], grad[1]) and torch.equal(got[n - 1], grad[0] + grad[2])
    assert got.count_nonzero() == got[5].count_nonzero() + got[n - 1].count_nonzero()


def test_logits_past_32_bits(gpu):
    batch, beams, vocab, top = 40, 64, 900_007, 8  # 4.6 GB
    logits = torch.zeros(batch, beams, vocab, device="cuda", dtype=torch.bfloat16)
    at = torch.randint(0, vocab, (batch, beams), generator=_gen(3), device="cuda")
    great = torch.randperm(batch * beams, generator=_gen(4), device="cuda").view(batch, beams) % 64 + 20.0
    logits.scatter_(2, at[:, :, None], great[:, :, None].bfloat16())
    scores = -torch.rand(batch, beams, generator=_gen(5), device="cuda")
    out, parents, tokens = gpu.beam_select(logits, top, scores)
    # a row's sum is vocab - 1 ones and one great exponential
    c = scores.double() + great.double() - torch.log(torch.exp(great.double()) + (vocab - 1))
    want = c.sort(dim=1, descending=True)
    assert torch.equal(parents.long(), want.indices[:, :top])
    assert torch.equal(tokens.long(), at.gather(1, want.indices[:, :top]))
    assert torch.all((out.double() - want.values[:, :top]).abs() <= 1e-5)


def test_odd_expert_rows_past_32_bits(gpu):
    experts, hidden, inner = 600, 2047, 2047  # 5 GB to each matrix
    up = torch.zeros(experts, inner, hidden, dtype=torch.float16, device="cuda")
    down = torch.zeros(experts, hidden, inner, dtype=torch.float16, device="cuda")
    up[-1, -1, -1], up[1, 7, 5], down[-1, -1, -1], down[1, 9, 7] = 2.0, 3.0, 4.0, 5.0
    x = torch.zeros(2, hidden, dtype=torch.float16, device="cuda")
    x[:, 5], x[:, -1] = 1.0, 1.0
    ids = torch.tensor([[experts - 1], [1]], dtype=torch.int32, device="cuda")
    got = gpu.expert_mlp(x, ids, torch.ones(2, 1, device="cuda"), up, down, act="relu")
    assert got[0, -1] == 8 and got[1, 9] == 15 and got.count_nonzero() == 2


class Ways:
    """Calls that take the kernels which small aligned ones do not."""

    def __init__(self, om, seed):
        self.om, gen = om, _gen(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.logits = rand(1, 3, 131071).half()                          # a cluster of sixteen
        self.states = rand(2, 20, 2, 9, 7)                               # through shared memory
        self.parents = torch.randint(0, 20, (2, 20), generator=gen, device="cuda", dtype=torch.int32)
        self.table = rand(500, 77)
        self.grads = [(rand(n, w).bfloat16(), torch.randint(-1, 500, (n,), generator=gen, device="cuda"))
                      for n, w in ((100, 77), (20_000, 64), (270_000, 8))]  # counted, one cluster, merged
        self.x, self.ids = rand(9, 63).half(), torch.randint(-1, 4, (9, 3), generator=gen, device="cuda", dtype=torch.int32)
        self.weights, self.up, self.down = rand(9, 3), (rand(4, 31, 63) / 8).half(), (rand(4, 63, 31) / 6).half()

    def __call__(self):
        om = self.om
        moved = self.states.clone()
        om.beam_gather(self.parents, (moved,))
        return [*om.beam_select(self.logits, 64), moved, om.embed_lookup(self.grads[0][1], self.table, 0.5),
                *(om.embed_lookup_backward(g, i, 500, 2.0) for g, i in self.grads),
                om.expert_mlp(self.x, self.ids, self.weights, self.up, self.down, gate=self.up, act="gelu")]

    def change(self, seed):
        for t in (self.logits, self.states, self.table, self.x, *(g for g, _ in self.grads)):
            t.normal_(generator=_gen(seed))


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_captured_on_every_way(gpu):
    ways = [Ways(gpu, 1), Ways(gpu, 2)]
    graphs, outs = [], []
    for w in ways:
        w()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w())
        graphs.append(graph)
    for seed in range(3):
        for w in ways:
            w.change(10 + seed)
        for graph in graphs:
            graph.replay()
        for w, out in zip(ways, outs):
            assert _same(out, w())
        for graph in reversed(graphs):
            graph.replay()
        torch.cuda.synchronize()
        for w, out in zip(ways, outs):
            assert _same(out, w())


def test_from_several_threads(gpu):
    """Each thread calls on a stream of its own, all at once; the first calls of each way may be among them."""
    ways = [Ways(gpu, i) for i in range(4)]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [ways[i]() for _ in range(6)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for w, each in zip(ways, got):
        want = w()
        assert all(_same(g, want) for g in each)
    assert gpu.device_error() == 0


def test_gradient_through_a_narrow_batch(gpu):
    """A padded batch: rows behind each sequence's end ask for no row, and their gradient counts for nothing."""
    gen = _gen(7)
    table = torch.randn(60, 33, generator=gen, device="cuda", requires_grad=True)
    ids = torch.randint(0, 60, (5, 40), generator=gen, device="cuda")
    for b, n in enumerate((40, 1, 0, 17, 39)):
        ids[b, n:] = -1
    pull = torch.randn(5, 40, 33, generator=gen, device="cuda")
    pull[ids < 0] = float("nan")
    rows = gpu.embed_lookup(ids, table, 3.0)
    assert not rows[ids < 0].any()
    grad, = torch.autograd.grad(rows, table, pull)
    want, error = ref.embed_backward(pull.nan_to_num(0.0), ids, 60, 3.0)
    assert torch.all((grad.double() - want).abs() <= error + 2 * ref.E32 * want.abs())
