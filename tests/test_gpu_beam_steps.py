"""Steps of a beam search as they come: the first, of one live beam, later ones with ended beams, and rows whose neighbours
in memory are no numbers."""
import pytest
import torch

from test_gpu_beam import _check, _logits, _moved

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,beams,vocab,top", [(1, 4, 131071, 8), (2, 8, 70001, 16), (1, 16, 65537, 32), (16, 5, 50021, 10),
                                                   (40, 9, 20011, 18), (300, 6, 5003, 12)])
def test_one_live_beam(gpu, dtype, batch, beams, vocab, top):
    """The first step's scores: all beams hold the same prompt, so one goes on; each time another."""
    logits, _ = _logits(batch, beams, vocab, dtype)
    scores = torch.full((batch, beams), -INF, device="cuda")
    at = torch.arange(batch, device="cuda") % beams
    scores[torch.arange(batch, device="cuda"), at] = -3.0
    out, parents, tokens = _check(gpu, logits, top, scores)
    assert torch.all(parents == at[:, None])
    # and with the others ended, not dead
    finished = scores == -INF
    scores[finished] = -40.0
    _check(gpu, logits, top, scores, finished, vocab - 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("beams", [3, 6, 9, 12])
def test_some_beams_ended(gpu, dtype, beams):
    for batch, vocab in ((2, 40009), (30, 9001)):
        logits, scores = _logits(batch, beams, vocab, dtype)
        gen = torch.Generator(device="cuda").manual_seed(beams)
        finished = torch.rand(batch, beams, generator=gen, device="cuda") < 0.5
        scores[torch.rand(batch, beams, generator=gen, device="cuda") < 0.2] = -INF
        logits[finished] = float("nan")
        _check(gpu, logits, 2 * beams, scores, finished, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("around", [float("nan"), INF, 60000.0])
def test_what_lies_around_the_rows_counts_for_nothing(gpu, dtype, around):
    """Whole 16 bytes around a row are read: greater values there, infinities and NaN, are none of the row's."""
    for vocab in (1, 5, 1003, 8193, 33001):
        for shift in range(8):
            apart = vocab + 1 + shift
            room = torch.full((2 * 3 * apart + 16,), around, device="cuda", dtype=dtype)
            rows = room[shift:shift + 6 * apart].view(2, 3, apart)[:, :, :vocab]
            rows.copy_(_logits(2, 3, vocab, dtype)[0])
            _check(gpu, rows, 7, torch.tensor([[-1.0, -2.0, -1.5], [-3.0, -3.0, -3.5]], device="cuda"))


@pytest.mark.parametrize("beams", [4, 8, 16, 17, 64])
@pytest.mark.parametrize("count", [4, 5, 64])
def test_many_states_at_once(gpu, beams, count):
    """Arrays of mixed sizes, as many as one launch carries, in place and into others, between starts and lengths."""
    gen = torch.Generator(device="cuda").manual_seed(beams * count)
    batch, heads, entries = 2, 2, 23
    tails = ((16,), (), (3,), (2, 5))
    types = (torch.bfloat16, torch.float32, torch.int8, torch.float16)
    new = lambda i: torch.randint(-100, 100, (batch, beams, heads, entries, *tails[i % 4]), generator=gen, device="cuda").to(types[i % 4])  # noqa: E731
    parents = torch.randint(-1, beams + 1, (batch, beams), generator=gen, device="cuda", dtype=torch.int32)
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([entries, 19], dtype=torch.int32, device="cuda")
    for lo, hi in ((None, None), (starts, lengths)):
        states, into = [new(i) for i in range(count)], [new(i) for i in range(count)]
        want = [_moved(s, parents, lo, hi) for s in states]
        elsewhere = [_moved(s, parents, lo, hi, o) for s, o in zip(states, into)]
        gpu.beam_gather(parents, states, starts=lo, lengths=hi, out=into)
        assert all(torch.equal(a, b) for a, b in zip(into, elsewhere))
        gpu.beam_gather(parents, states, starts=lo, lengths=hi)
        assert all(torch.equal(a, b) for a, b in zip(states, want))


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_of_rows_among_no_numbers(gpu, dtype):
    ids = torch.tensor([3, -1, 0, 6, 6, 2, 7, 5], device="cuda")
    for width in (1, 5, 8, 33, 127, 1025):
        for shift in range(8):
            apart = width + 1 + shift
            room = torch.full((7 * apart + 16,), float("nan"), device="cuda", dtype=dtype)
            table = room[shift:shift + 7 * apart].view(7, apart)[:, :width]
            table.copy_(torch.randn(7, width, device="cuda"))
            got = gpu.embed_lookup(ids, table, 0.5)
            want = torch.where(((ids >= 0) & (ids < 7))[:, None], (table[ids.clamp(0, 6)].float() * 0.5).to(dtype), 0.0)
            assert torch.equal(got, want)
