"""Beam search, embedding rows and routed experts as programs meet them: captured in graphs, on several streams,
with autograd's graph alive, on another stream than the data's."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu


class Step:
    """One decoding step's calls on tensors of its own."""

    def __init__(self, om, seed, batch=2, beams=4, vocab=5003):
        self.om, gen = om, torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.gen, self.batch, self.beams = gen, batch, beams
        self.logits, self.scores = rand(batch, beams, vocab).bfloat16(), -rand(batch, beams).abs()
        self.finished = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
        self.cache = rand(batch, beams, 2, 40, 32).bfloat16()
        self.table, self.grad = rand(vocab, 128).bfloat16(), rand(900, 128).bfloat16()
        self.ids = torch.randint(-1, vocab, (900,), generator=gen, device="cuda")
        mat = lambda *s: (rand(*s) * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.router, self.up, self.gate, self.down = mat(32, 128), mat(32, 72, 128), mat(32, 72, 128), mat(32, 128, 72)

    def __call__(self):
        om = self.om
        scores, parents, tokens = om.beam_select(self.logits, self.beams, self.scores, finished=self.finished, end_id=2)
        moved = self.cache.clone()
        om.beam_gather(parents, (moved,))
        x = om.embed_lookup(tokens, self.table, 2.0).flatten(0, 1)
        ids, w = om.route_topk(x @ self.router.t(), 4, renorm=True)
        y = om.expert_mlp(x, ids, w, self.up, self.down, gate=self.gate)
        grad = om.embed_lookup_backward(self.grad, self.ids, len(self.table))
        more = om.embed_lookup_backward(self.grad, self.ids % 40, len(self.table), 0.5, True, grad.clone())
        return scores, parents, tokens, moved, x, y, grad, more

    def change(self, seed):
        self.gen.manual_seed(seed)
        for t in (self.logits, self.cache, self.table, self.grad):
            t.normal_(generator=self.gen)
        self.ids.random_(-1, len(self.table), generator=self.gen)


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs(gpu):
    """Two captured steps, replayed in turn and with eager calls between: no scratch of one is the other's."""
    steps = [Step(gpu, 1), Step(gpu, 2, batch=3, beams=2, vocab=301)]
    graphs, outs = [], []
    for s in steps:
        s()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s()
        graphs.append(graph)
        outs.append(out)
    for seed in range(3):
        for s in steps:
            s.change(seed)
        for graph in graphs:
            graph.replay()
        between = steps[0]()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], between)
        for s, out in zip(steps, outs):
            assert _same(out, s())


def test_streams_at_once(gpu):
    """Steps issued on four streams without a wait between."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    steps = [Step(gpu, i) for i in range(4)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    got = [[] for _ in steps]
    for _ in range(5):
        for i, (s, stream) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(stream):
                got[i].append(s())
    torch.cuda.synchronize()
    assert all(_same(g, want[i]) for i in range(4) for g in got[i])
    assert gpu.device_error() == 0


def test_inputs_written_just_before(gpu):
    """Calls right behind the kernels that write their inputs (a launch may start while the one before drains)."""
    s = Step(gpu, 5)
    for seed in range(10):
        s.change(100 + seed)
        got = s()
        torch.cuda.synchronize()
        assert _same(got, s())


def test_backward_in_a_graph(gpu):
    """A training step's gradient captured and replayed; autograd's graph of an eager step is gone by then."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randn(77, 24, generator=gen, device="cuda").requires_grad_()
    ids = torch.randint(0, 77, (3, 50), generator=gen, device="cuda")
    pull = torch.randn(3, 50, 24, generator=gen, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            grad, = torch.autograd.grad((gpu.embed_lookup(ids, table) * pull).sum(), table)
    torch.cuda.current_stream().wait_stream(side)
    del grad
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad, = torch.autograd.grad((gpu.embed_lookup(ids, table) * pull).sum(), table)
    for seed in range(3):
        ids.random_(-5, 77, generator=gen)
        pull.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        want, error = ref.embed_backward(pull, ids, 77)
        assert torch.all((grad.double() - want).abs() <= error + 2 * ref.E32 * want.abs())


def test_library_allocates_no_torch_memory_but_outputs(gpu):
    """Outputs handed in: no call allocates through torch."""
    s = Step(gpu, 7)
    out = [torch.empty(2, 4, device="cuda"), torch.empty(2, 4, dtype=torch.int32, device="cuda"), torch.empty(2, 4, dtype=torch.int32, device="cuda")]
    x = torch.randn(8, 128, device="cuda").bfloat16()
    ids, w = gpu.route_topk(x @ s.router.t(), 4)
    y, rows, table = torch.empty_like(x), torch.empty(900, 128, device="cuda").bfloat16(), torch.empty_like(s.table)
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    gpu.beam_select(s.logits, 4, s.scores, out_scores=out[0], parents=out[1], tokens=out[2])
    gpu.beam_gather(out[1], (s.cache,))
    gpu.embed_lookup(s.ids, s.table, out=rows)
    gpu.embed_lookup_backward(s.grad, s.ids, len(table), grad_table=table)
    gpu.expert_mlp(x, ids, w, s.up, s.down, gate=s.gate, out=y)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_refusals_on_the_gpu(gpu):
    s = Step(gpu, 8)
    x = torch.randn(65, 128, device="cuda").bfloat16()
    ids, w = gpu.route_topk(x @ s.router.t(), 4)
    for call in (lambda: gpu.beam_select(s.logits, 65), lambda: gpu.beam_select(s.logits, 0),
                 lambda: gpu.beam_select(s.logits, 4, finished=s.finished, end_id=5003),
                 lambda: gpu.expert_mlp(x, ids, w, s.up, s.down), lambda: gpu.expert_mlp(x[:4], ids[:4], w[:4], s.up, s.down, out=x[:4]),
                 lambda: gpu.embed_lookup(s.ids, s.table, out=s.table[:900])):
        with pytest.raises(gpu.OrdMergeError):
            call()
    for call in (lambda: gpu.beam_gather(torch.zeros(2, 4, dtype=torch.int32, device="cuda"), (s.cache, s.cache[:, :, :1])),
                 lambda: gpu.embed_lookup(s.ids.cpu(), s.table), lambda: gpu.expert_mlp(x[:4], ids[:4], w[:4], s.up, s.down.cpu())):
        with pytest.raises(ValueError):
            call()
    for v in gpu.beam_select(s.logits[:0], 4):
        assert v.shape == (0, 4)
    assert gpu.expert_mlp(x[:0], ids[:0], w[:0], s.up, s.down).shape == (0, 128)
    assert gpu.embed_lookup_backward(s.grad[:0], s.ids[:0], 7).shape == (7, 128)
