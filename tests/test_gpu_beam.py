"""om_beam_select and om_beam_gather against their definitions in 64 bits."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def _logits(batch, beams, vocab, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + vocab)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return (rand(batch, beams, vocab) * 3).to(dtype), -rand(batch, beams).abs() * 2 - 3


def _check(om, logits, top, scores=None, finished=None, end_id=0):
    got = om.beam_select(logits, top, scores, finished=finished, end_id=end_id)
    ref.check_beams(got, logits, top, scores, finished, end_id)
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 127, 511, 4096, 4099, 20011, 50021, 131071])
def test_select_sizes(gpu, dtype, vocab):
    for batch, beams, top in ((1, 1, 1), (1, 4, 8), (2, 3, 6), (3, 5, 64)):
        logits, scores = _logits(batch, beams, vocab, dtype)
        _check(gpu, logits, top, scores)


@pytest.mark.parametrize("batch,beams,top", [(1, 64, 64), (1, 17, 3), (40, 16, 32), (200, 7, 14), (700, 2, 4), (5, 33, 64)])
def test_select_shapes(gpu, batch, beams, top):
    logits, scores = _logits(batch, beams, 3001, torch.bfloat16)
    _check(gpu, logits, top, scores)


@pytest.mark.parametrize("batch,beams,vocab,top", [(1, 16, 131071, 32), (1, 3, 131072, 6), (4, 8, 70001, 16), (5, 8, 70001, 16),
                                                   (2, 5, 60000, 10), (1, 64, 20011, 64), (1, 1, 400003, 5)])
def test_select_few_sequences(gpu, batch, beams, vocab, top):
    """Shapes on both sides of the rule for wide clusters."""
    for dtype in (torch.float32, torch.bfloat16):
        logits, scores = _logits(batch, beams, vocab, dtype)
        _check(gpu, logits, top, scores)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_no_scores_is_greedy_choice(gpu, dtype):
    logits, _ = _logits(9, 1, 32001, dtype)
    out, parents, tokens = _check(gpu, logits, 1)
    assert torch.equal(tokens[:, 0].long(), logits[:, 0].float().cpu().sort(dim=1, descending=True, stable=True).indices[:, 0].cuda())
    assert int(parents.max()) == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [9, 300, 5003, 131071])
def test_equal_rows_tie_to_the_lower_beam(gpu, dtype, vocab):
    """Rows of the same values, each at another address modulo 16: every continuation ties with the other beams'."""
    one, _ = _logits(1, 1, vocab, dtype)
    logits = one.expand(2, 8, vocab).contiguous()
    out, parents, tokens = _check(gpu, logits, 16, torch.full((2, 8), -4.0, device="cuda"))
    order = one[0, 0].float().cpu().sort(descending=True, stable=True).indices
    # equal logits of a row come beam by beam: sort by (logit, beam, token)
    x = one[0, 0].float().cpu()
    flat = sorted(((-float(x[t]), i, int(t)) for t in order[:16] for i in range(8)))[:16]
    for b in range(2):
        assert [(i, t) for _, i, t in flat] == list(zip(parents[b].tolist(), tokens[b].tolist()))


@pytest.mark.parametrize("dtype", TYPES)
def test_constant_and_nearly_constant_rows(gpu, dtype):
    """Rows of one value, and of the type's lowest value with a few others: more candidates than the kernel has room for."""
    for vocab in (1000, 40009):
        logits = torch.zeros(2, 3, vocab, dtype=dtype, device="cuda")
        logits[1] = -2.5
        scores = torch.tensor([[-1.0, -2.0, -1.5], [-3.0, -3.0, -3.0]], device="cuda")
        out, parents, tokens = _check(gpu, logits, 6, scores)
        assert parents.tolist() == [[0] * 6, [0] * 6] and tokens.tolist() == [list(range(6))] * 2
        masked = torch.full((2, 3, vocab), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        masked[:, :, 37] = 1.5
        masked[0, 1, 900] = 2.0
        out, parents, tokens = _check(gpu, masked, 8, scores)
        assert (parents[0, 0], tokens[0, 0]) == (0, 37)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", ["lowest", 0.0, -1e9])
def test_few_logits_above_many_equal_ones(gpu, dtype, low):
    """A grammar's few tokens, all others at one value: the first of these fill up, wherever they are."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    for vocab, top in ((2000, 8), (70001, 20), (131071, 64)):
        logits = torch.full((3, 2, vocab), low, device="cuda").to(dtype)  # (-1e9 is -inf in 16 bits with 5 of exponent)
        for b in range(3):
            at = torch.randperm(vocab, generator=torch.Generator(device="cuda").manual_seed(b), device="cuda")[:5 * b + 1]
            logits[b, :, at] = torch.arange(5.0 * b + 1, device="cuda").to(dtype) + 1
        logits[2, 0, :vocab // 2] = -INF
        logits[1, 1, :600] = float("nan")
        _check(gpu, logits, top, torch.tensor([[-1.0, -1.25], [-2.0, -1.0], [-1.0, -1.0]], device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
def test_great_logits_at_a_regular_distance(gpu, dtype):
    """More great logits than candidates have room, all in the words of a few threads, so that the bound is low."""
    vocab = 30001
    logits, scores = _logits(3, 16, vocab, dtype)
    word = torch.arange(vocab, device="cuda") // (1 if dtype == torch.float32 else 2)
    for few in (3, 10, 30):
        great = word % 256 < few
        x = torch.where(great, logits + 100, logits)
        _check(gpu, x, 64, scores)
        x[0, 3] = torch.where(great, 50.0, -50.0).to(dtype)
        _check(gpu, x, 64, scores)


@pytest.mark.parametrize("dtype", TYPES)
def test_ascending_rows(gpu, dtype):
    """The greatest logits all at the end, in one thread's part, and equal in groups."""
    ramp = (torch.arange(30011, device="cuda") // 7).float() / 400
    logits = torch.stack([ramp, ramp.flip(0), ramp])[None].to(dtype)
    _check(gpu, logits, 40, torch.tensor([[-1.0, -1.5, -1.25]], device="cuda"))
    block = torch.zeros(1, 1, 60000, device="cuda")
    block[..., 4096:4104] = torch.arange(8.0, device="cuda")  # one vector holds them all
    _check(gpu, block.to(dtype), 8)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [12, 1001, 33000])
def test_masked_logits(gpu, dtype, vocab):
    logits, scores = _logits(4, 3, vocab, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    hide = torch.rand(logits.shape, generator=gen, device="cuda")
    logits[hide < 0.4] = -INF
    logits[hide > 0.9] = float("nan")
    logits[1, 0] = -INF                  # a row with nothing
    logits[2] = -INF                     # a sequence with nothing
    logits[3, :, 5:] = float("nan")      # a handful left
    logits[3, :, :5] = torch.arange(5.0, device="cuda").to(dtype)
    out, parents, tokens = _check(gpu, logits, 20, scores)
    assert torch.all(parents[2] == -1) and torch.all(parents[3, 15:] == -1) and torch.all(parents[3, :15] >= 0)


def test_large_logits(gpu):
    """Magnitudes at which a product with log2 e rounds to more than a step of the sum, and the greatest of all."""
    for size in (1e3, 9.9e5, 1.1e6, 1e20, 1e38):
        logits, scores = _logits(2, 3, 5001, torch.float32)
        _check(gpu, logits / 12 * size, 6, scores)
        _check(gpu, logits + size, 6, scores)
        _check(gpu, logits - size, 6, scores)
        logits[:, :, 3000:] = -torch.finfo(torch.float32).max
        _check(gpu, logits + size, 6, scores)


def test_infinite_logits_and_scores(gpu):
    logits, scores = _logits(3, 4, 777, torch.float32)
    logits[0, 1, 5] = INF                # no finite probabilities: no continuation
    scores[0, 2] = -INF                  # beams that do not go on
    scores[1, :] = float("nan")
    scores[2, 0], scores[2, 3] = float("nan"), -INF
    logits[2, 1] *= 1e30                 # far apart, no overflow
    out, parents, tokens = _check(gpu, logits, 9, scores)
    assert not {1, 2} & set(parents[0].tolist()) and torch.all(parents[1] == -1) and not {0, 3} & set(parents[2].tolist())


@pytest.mark.parametrize("dtype", TYPES)
def test_finished_beams(gpu, dtype):
    logits, scores = _logits(3, 4, 5001, dtype)
    finished = torch.tensor([[0, 1, 0, 0], [1, 1, 1, 1], [1, 0, 0, 1]], dtype=torch.bool, device="cuda")
    scores[2, 3] = -INF                  # finished and dead
    logits[0, 1] = float("nan")          # not read
    out, parents, tokens = _check(gpu, logits, 6, scores, finished, 77)
    assert sorted(parents[1, :4].tolist()) == [0, 1, 2, 3] and tokens[1].tolist() == [77] * 4 + [-1, -1]
    assert torch.equal(out[1, :4], scores[1].sort(descending=True).values)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_strides_and_alignment(gpu, dtype):
    """Rows of any address, rows apart, overlapping rows (one row for all beams) and rows at the end of memory."""
    for shift in range(8):
        buf = torch.randn(4 * 3 * 1100 + 16, device="cuda").to(dtype)
        view = buf[shift:shift + 4 * 3 * 1100].view(4, 3, 1100)
        _check(gpu, view[:, :, :1003], 7)
        _check(gpu, view[1:, 1:, shift:1003], 7)
        _check(gpu, view[:, :1, 3:900].expand(4, 5, 897), 7)


def test_select_on_a_stream_and_repeated(gpu):
    logits, scores = _logits(8, 6, 65537, torch.bfloat16)
    want = gpu.beam_select(logits, 12, scores)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine = logits + 0
    for _ in range(3):
        got = gpu.beam_select(mine, 12, scores, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- gather --

def _moved(x, parents, starts, lengths, into=None):
    out = (x if into is None else into).clone()
    batch, beams, _, entries = x.shape[:4]
    for b in range(batch):
        lo = 0 if starts is None else max(0, int(starts[b]))
        hi = entries if lengths is None else min(entries, int(lengths[b]))
        for j in range(beams):
            p = int(parents[b, j])
            if 0 <= p < beams and lo < hi:
                out[b, j, :, lo:hi] = x[b, p, :, lo:hi]
    return out


def _states(batch, beams, heads, entries, gen):
    rand = lambda *s: torch.randint(-128, 127, s, generator=gen, device="cuda")  # noqa: E731
    return [rand(batch, beams, heads, entries, 64).to(torch.bfloat16), rand(batch, beams, heads, entries, 3).to(torch.int8),
            rand(batch, beams, heads, entries).float(), rand(batch, beams, heads, entries, 2, 9).to(torch.float16)]


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 9, 16, 17, 40, 64])
@pytest.mark.parametrize("entries", [1, 37, 300])
def test_gather_in_place_and_elsewhere(gpu, beams, entries):
    gen = torch.Generator(device="cuda").manual_seed(beams * entries)
    batch, heads = 3, 2
    for kind in range(4):
        parents = torch.randint(-1 if kind else 0, beams, (batch, beams), generator=gen, device="cuda", dtype=torch.int32)
        if kind == 2:
            parents[:] = torch.arange(beams, device="cuda").roll(1)  # one cycle
        if kind == 3:
            parents[0], parents[1, 0], parents[2, -1] = 0, beams, -(1 << 31)
        starts = torch.tensor([0, entries // 3, entries + 5], device="cuda", dtype=torch.int32) if kind else None
        lengths = torch.tensor([entries, entries // 2, entries], device="cuda", dtype=torch.int32) if kind != 2 else None
        states = _states(batch, beams, heads, entries, gen)
        into = [torch.full_like(s, 5) for s in states]
        want = [_moved(s, parents, starts, lengths) for s in states]
        elsewhere = [_moved(s, parents, starts, lengths, o) for s, o in zip(states, into)]
        got = gpu.beam_gather(parents, states, starts=starts, lengths=lengths, out=into)
        assert all(torch.equal(a, b) for a, b in zip(got, elsewhere))
        got = gpu.beam_gather(parents, states, starts=starts, lengths=lengths)
        assert all(a is b for a, b in zip(got, states))
        assert all(torch.equal(a, b) for a, b in zip(states, want))


def test_gather_lengths_out_of_range(gpu):
    x = torch.arange(2 * 3 * 10, device="cuda").view(2, 3, 1, 10)
    parents = torch.tensor([[2, 0, 1], [1, 1, 1]], device="cuda", dtype=torch.int32)
    for lo, hi in ((-7, 99), (4, 4), (6, 2), (2 ** 31 - 1, -2 ** 31), (-2 ** 31, 2 ** 31 - 1)):
        starts, lengths = (torch.full((2,), v, device="cuda", dtype=torch.int32) for v in (lo, hi))
        y = x.clone()
        gpu.beam_gather(parents, (y,), starts=starts, lengths=lengths)
        assert torch.equal(y, _moved(x, parents, starts, lengths))


@pytest.mark.parametrize("beams", [4, 20])
def test_gather_strided_caches(gpu, beams):
    """Keys beside values in one buffer, heads last but one, a part of a greater cache, and rows of odd addresses."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    parents = torch.randint(0, beams, (2, beams), generator=gen, device="cuda", dtype=torch.int32)
    both = torch.randint(0, 99, (2, beams, 2, 3, 50, 32), generator=gen, device="cuda").half()
    k, v = both[:, :, 0], both[:, :, 1]
    want = [_moved(x, parents, None, None) for x in (k, v)]
    gpu.beam_gather(parents, (k, v))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    late = torch.randint(0, 99, (2, beams, 50, 3, 32), generator=gen, device="cuda").float().transpose(2, 3)
    want = _moved(late, parents, None, None)
    gpu.beam_gather(parents, (late,))
    assert torch.equal(late, want)
    big = torch.randint(0, 99, (2, beams, 4, 80, 33), generator=gen, device="cuda").half()
    before, part = big.clone(), big[:, :, 1:3, 5:60, 1:]
    want = _moved(part, parents, None, None)
    gpu.beam_gather(parents, (part,))
    assert torch.equal(part, want)
    part.copy_(before[:, :, 1:3, 5:60, 1:])
    assert torch.equal(big, before)  # nothing beside it was touched


def test_gather_many_arrays(gpu):
    gen = torch.Generator(device="cuda").manual_seed(8)
    parents = torch.randint(0, 4, (2, 4), generator=gen, device="cuda", dtype=torch.int32)
    layers = [torch.randn(2, 4, 2, 20, 16, generator=gen, device="cuda") for _ in range(64)]
    want = [_moved(x, parents, None, None) for x in layers]
    gpu.beam_gather(parents, layers)
    assert all(torch.equal(a, b) for a, b in zip(layers, want))
    with pytest.raises(gpu.OrdMergeError):
        gpu.beam_gather(parents, layers + [torch.zeros_like(layers[0])])
    with pytest.raises(gpu.OrdMergeError):  # into a part of itself
        x = torch.zeros(2, 4, 1, 30, 16, device="cuda")
        gpu.beam_gather(parents, (x[:, :, :, :20],), out=(x[:, :, :, 10:],))


def test_gather_offsets_past_32_bits(gpu):
    """A cache of more than 4 GB: beams 2.2 GB apart."""
    x = torch.zeros(1, 3, 1, 1 << 24, 66, dtype=torch.int16, device="cuda")
    for j in range(3):
        x[0, j, 0, -5:] = j + 1
        x[0, j, 0, :5] = j + 11
    parents = torch.tensor([[2, 2, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([(1 << 24) - 1], dtype=torch.int32, device="cuda")
    gpu.beam_gather(parents, (x,), lengths=lengths)
    assert x[0, :, 0, 0, 0].tolist() == [13, 13, 11] and x[0, :, 0, -2, 65].tolist() == [3, 3, 1]
    assert x[0, :, 0, -1, 0].tolist() == [1, 2, 3]
