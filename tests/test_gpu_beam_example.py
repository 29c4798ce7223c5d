"""The beam-search example: its calls together, each checked as it is made, and its training gradient."""
import importlib.util
import os

import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("beam_decode", os.path.join(ROOT, "examples", "beam_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Checked:
    """The package, with each call of a decoding step compared with its definition."""

    def __init__(self, om):
        self.om, self.calls = om, {}

    def __getattr__(self, name):
        return getattr(self.om, name)

    def _count(self, name):
        self.calls[name] = self.calls.get(name, 0) + 1

    def beam_select(self, logits, top, scores=None, finished=None, end_id=0):
        got = self.om.beam_select(logits, top, scores, finished=finished, end_id=end_id)
        ref.check_beams(got, logits, top, scores, finished, end_id)
        self._count("beam_select")
        return got

    def beam_gather(self, parents, arrays, starts=None, lengths=None):
        before = [a.clone() for a in arrays]
        self.om.beam_gather(parents, arrays, starts=starts, lengths=lengths)
        for a, x in zip(arrays, before):
            for b in range(a.shape[0]):
                lo, hi = int(starts[b]), int(lengths[b])
                want = x[b].clone()
                want[:, :, lo:hi] = x[b, parents[b].long(), :, lo:hi]
                assert torch.equal(a[b], want)
        self._count("beam_gather")
        return arrays

    def embed_lookup(self, ids, table, scale=1.0):
        got = self.om.embed_lookup(ids, table, scale)
        with torch.no_grad():
            assert torch.equal(got, (table[ids.long()].float() * scale).to(table.dtype))
        self._count("embed_lookup")
        return got

    def expert_mlp(self, x, ids, weights, up, down, gate=None, act="silu"):
        got = self.om.expert_mlp(x, ids, weights, up, down, gate=gate, act=act)
        ref.DT[0] = x.dtype
        want, error = ref.expert_mlp(x, ids, weights, up, down, gate, act)
        assert torch.all((got.double() - want).abs() <= error + ref.HALF[got.dtype] * (want.abs() + error) + 2.0 ** -25)
        self._count("expert_mlp")
        return got


def test_steps_of_a_beam_search(gpu, example, monkeypatch):
    torch.manual_seed(1)
    checked = Checked(gpu)
    monkeypatch.setattr(example, "om", checked)
    model = example.Model(vocab=301, hidden=64, heads=2, experts=8, inner=32, picks=2)
    prompts = torch.randint(3, 301, (3, 4), device="cuda")
    tokens, scores = example.beam_search(model, prompts, beams=5, steps=6, end_id=2)
    assert tokens.shape == (3, 5, 6) and torch.all(scores[:, 1:] <= scores[:, :-1])
    assert checked.calls == {"beam_select": 6, "beam_gather": 5, "embed_lookup": 9, "expert_mlp": 9}
    # each sequence's score is the sum of its tokens' log probabilities, stepped through on its own
    monkeypatch.setattr(example, "om", gpu)
    for b in range(3):
        for j in (0, 4):
            cache, total, ended = model.caches(1, 1, 10), 0.0, False
            path = [*prompts[b].tolist(), *tokens[b, j].tolist()]
            for i, t in enumerate(path[:-1]):
                logits = model.step(torch.tensor([[t]], device="cuda"), cache, i)
                if i >= 3 and not ended:
                    total += float(logits[0, 0].double().log_softmax(0)[path[i + 1]])
                    ended = path[i + 1] == 2
            # 16-bit products of other shapes run in another order: a step of the logits (about 8 at most) each
            assert abs(total - float(scores[b, j])) <= 6 * 8 * 2 * ref.HALF[torch.bfloat16]


def test_training_gradient(gpu, example):
    gen = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randn(50, 16, generator=gen, device="cuda").requires_grad_()
    out = torch.randn(16, 50, generator=gen, device="cuda")
    tokens = torch.randint(0, 50, (4, 9), generator=gen, device="cuda")
    grad, = torch.autograd.grad(example.next_token_loss(table, out, tokens), table)
    t64 = table.detach().double().requires_grad_()
    loss = torch.nn.functional.cross_entropy((t64[tokens[:, :-1]] @ out.double()).flatten(0, 1), tokens[:, 1:].flatten())
    want, = torch.autograd.grad(loss, t64)
    # products of 16 and 50 terms in 32 bits, a softmax of arguments up to 30, sums of a few rows
    assert (grad - want).abs().max() <= (16 + 50 + 60 + 40) * ref.E32 * 30 * want.abs().max()


def test_example_runs(gpu, example, capsys):
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert sum(line.startswith("prompt") for line in lines) == 3 and sum(line.startswith("step") for line in lines) == 3
