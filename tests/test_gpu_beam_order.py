"""The order of a beam search's continuations where their scores round to one number: beam by beam, and within a beam
by logit, then token, however many slices a row is cut into."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
LOWEST = -torch.finfo(torch.float32).max


def _expected(logits, scores, top, margin=0.0):
    """parents and tokens [batch, top]; a score's rounding may not hang on the last places of a logarithm."""
    x = logits.double().cpu()
    lse = torch.logsumexp(x, 2, keepdim=True)
    p = scores.double().cpu()[:, :, None]
    c = p + (x - lse)
    if margin:
        assert torch.equal(c, p + (x - lse + margin)) and torch.equal(c, p + (x - lse - margin))
    beams, vocab = x.shape[1:]
    beam, token = np.divmod(np.arange(beams * vocab), vocab)
    out = [np.lexsort((token, -x[b].flatten().numpy(), beam, -c[b].flatten().numpy()))[:top] for b in range(len(x))]
    at = torch.from_numpy(np.stack(out))
    return at // vocab, at % vocab


def _check(om, logits, scores, top, margin=0.0):
    out, parents, tokens = (t.cpu() for t in om.beam_select(logits, top, scores))
    want = _expected(logits, scores, top, margin)
    assert torch.equal(parents.long(), want[0])
    assert torch.equal(tokens.long(), want[1])
    assert torch.equal(out, scores.cpu().gather(1, parents.long()))  # what a score's rounding leaves of it


# rows cut into eight, two and four slices, joined by counting and by taking; rows that are not cut
SHAPES = [(1, 1, 131071, 8), (1, 1, 131071, 64), (1, 3, 33000, 16), (1, 4, 70001, 40), (2, 2, 50021, 12), (7, 3, 33000, 64),
          (40, 8, 5003, 16), (400, 4, 3001, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", [-1e19, -1e30, LOWEST])
@pytest.mark.parametrize("batch,beams,vocab,top", SHAPES)
def test_scores_that_swallow_the_logits(gpu, dtype, score, batch, beams, vocab, top):
    gen = torch.Generator(device="cuda").manual_seed(vocab + top)
    logits = (torch.randn(batch, beams, vocab, generator=gen, device="cuda") * 3).to(dtype)
    scores = torch.full((batch, beams), score, device="cuda")
    _check(gpu, logits, scores, top)
    if beams > 1:  # the second beam before the first; the others behind them
        scores[:, 1] = score / 2
        _check(gpu, logits, scores, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,beams,vocab,top", SHAPES[:6])
def test_scores_that_round_logits_together(gpu, dtype, batch, beams, vocab, top):
    """At -1e16 a score's last place is 2: whole logits fall together by twos.  Many of each, so that slices tie."""
    gen = torch.Generator(device="cuda").manual_seed(vocab + top)
    logits = torch.randint(0, 12, (batch, beams, vocab), generator=gen, device="cuda").to(dtype)
    logits[:, :, 17::1000] = 12.0
    scores = torch.full((batch, beams), -1e16, device="cuda")
    out, parents, tokens = (t.cpu() for t in gpu.beam_select(logits, top, scores))
    want = _expected(logits, scores, top, 1e-4)
    assert torch.equal(parents.long(), want[0])
    assert torch.equal(tokens.long(), want[1])


@pytest.mark.parametrize("score", [-2.0, -1e17, LOWEST])
def test_the_choice_does_not_hang_on_the_cut(gpu, score):
    """The same two beams as the only sequence, as one of two hundred, and beside six beams that have ended."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    one = torch.randn(1, 2, 60000, generator=gen, device="cuda") * 2
    scores = torch.tensor([[score, score * 1.5 if score > -1e30 else score]], device="cuda")
    want = gpu.beam_select(one, 20, scores)
    many = gpu.beam_select(one.expand(200, 2, 60000), 20, scores.expand(200, 2).contiguous())
    eight = gpu.beam_select(one[:, [0, 1, 0, 0, 0, 0, 0, 0]], 20,
                            torch.cat([scores, torch.full((1, 6), -float("inf"), device="cuda")], 1))
    for got in (many, eight):
        for i in (1, 2):
            assert torch.all(got[i] == want[i])


@pytest.mark.parametrize("dtype", TYPES)
def test_ended_beams_among_swallowed_ones(gpu, dtype):
    """An ended beam's one continuation ties with the others' by beam."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    logits = (torch.randn(1, 3, 40000, generator=gen, device="cuda") * 3).to(dtype)
    scores = torch.full((1, 3), -1e19, device="cuda")
    finished = torch.tensor([[True, False, False]], device="cuda")
    out, parents, tokens = gpu.beam_select(logits, 9, scores, finished=finished, end_id=5)
    best = logits[0, 1].float().sort(descending=True, stable=True).indices[:8].tolist()
    assert parents[0].tolist() == [0] + [1] * 8 and tokens[0].tolist() == [5] + best
    finished = torch.tensor([[False, True, False]], device="cuda")
    out, parents, tokens = gpu.beam_select(logits[:, :, :6].contiguous(), 9, scores, finished=finished, end_id=5)
    order = [logits[0, i, :6].float().sort(descending=True, stable=True).indices.tolist() for i in (0, 2)]
    assert parents[0].tolist() == [0] * 6 + [1] + [2] * 2 and tokens[0].tolist() == order[0] + [5] + order[1][:2]
