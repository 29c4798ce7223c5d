"""om_accumulate_weights, om_evict_select and om_evict_gather against plain references."""
import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import DTYPES, U32, f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- accumulated weights --

def _accumulate_check(om, w, score, lengths, decay, kv_heads, **kw):
    got = om.accumulate_weights(w, score, lengths=lengths, decay=decay, kv_heads=kv_heads, **kw)
    b, hq, q, s = w.shape
    n = np.full(b, s) if lengths is None else np.clip(lengths.cpu().numpy(), 0, s)
    x = f64(w)
    for i in range(b):
        rows = x[i, :, :, :n[i]].reshape(kv_heads, hq // kv_heads * q, n[i])
        old = np.zeros((kv_heads, n[i])) if score is None else f64(score)[i, :, :n[i]] * float(np.float32(decay))
        want, size = rows.sum(1) + old, np.abs(rows).sum(1) + np.abs(old)
        # any order of adding m + 1 terms: at most m + 1 half ulps of the terms' sizes, one more for decay * score
        assert np.all(np.abs(f64(got)[i, :, :n[i]] - want) <= (rows.shape[1] + 2) * U32 * size)
        assert not got[i, :, n[i]:].any()
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (2, 4, 2, 1, 33), (3, 8, 8, 1, 1000), (2, 16, 2, 5, 257), (1, 6, 2, 64, 4099),
                                   (1, 2, 1, 1, 70001), (4, 8, 1, 3, 520), (1, 4, 1, 200, 96)], ids=str)
def test_accumulate_matches_reference(gpu, dtype, shape):
    b, hq, h, q, s = shape
    gen = torch.Generator(device="cuda").manual_seed(s)
    w = torch.rand(b, hq, q, s, generator=gen, device="cuda").to(DTYPES[dtype])
    score = torch.randn(b, h, s, generator=gen, device="cuda")
    lengths = torch.tensor([[s, 0, 1, s + 5, -3][i % 5] for i in range(b)], dtype=torch.int32, device="cuda")
    _accumulate_check(gpu, w, score, None, 1.0, h)
    _accumulate_check(gpu, w, score, lengths, 0.9, h)
    _accumulate_check(gpu, w, None, lengths, 1.0, h)


def test_accumulate_past_the_length_is_not_read(gpu):
    w = torch.rand(2, 4, 3, 90, device="cuda")
    score = torch.rand(2, 2, 90, device="cuda")
    n = torch.tensor([41, 64], dtype=torch.int32, device="cuda")
    want = gpu.accumulate_weights(w, score, lengths=n)
    for i in range(2):
        w[i, :, :, n[i]:] = float("nan")
        score[i, :, n[i]:] = float("inf")
    assert torch.equal(gpu.accumulate_weights(w, score, lengths=n), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_accumulate_strides_and_in_place(gpu, dtype):
    base = torch.rand(3, 12, 7, 611, device="cuda").to(DTYPES[dtype])
    for lo, hi in ((0, 611), (1, 610), (3, 300), (8, 520)):
        w = base[:, 2:10, 1:6, lo:hi]
        score = torch.rand(3, 9, 700, device="cuda")[:, 4:6, 5:5 + hi - lo]
        _accumulate_check(gpu, w, score, None, 0.5, 2)
        want = gpu.accumulate_weights(w, score, decay=0.5)
        got = gpu.accumulate_weights(w, score, decay=0.5, out=score)
        assert got.data_ptr() == score.data_ptr() and torch.equal(got, want)
    turned = base.transpose(1, 2)[:, :, :6]  # queries outside heads
    _accumulate_check(gpu, turned, None, None, 1.0, 7)
    _accumulate_check(gpu, base[:, :, :0], torch.rand(3, 4, 611, device="cuda"), None, 0.5, 4)  # no queries


def test_accumulate_repeats_bit_for_bit(gpu):
    w = torch.rand(2, 16, 33, 3001, device="cuda").half()
    first = gpu.accumulate_weights(w, kv_heads=4)
    for _ in range(4):
        assert torch.equal(gpu.accumulate_weights(w, kv_heads=4), first)


# ------------------------------------------------------------------ selection --

def _select_check(om, score, budget, first=0, last=0, lengths=None):
    keep, kept = om.evict_select(score, budget, first=first, last=last, lengths=lengths)
    n = np.full(score.shape[0], score.shape[2]) if lengths is None else lengths.cpu().numpy()
    want, wkept = ref.evict(score.cpu().numpy(), n, budget, first, last)
    assert np.array_equal(keep.cpu().numpy(), want)
    assert np.array_equal(kept.cpu().numpy(), wkept)
    return keep


@pytest.mark.parametrize("length", [1, 2, 63, 64, 1000, 1025, 4096, 30001])
@pytest.mark.parametrize("batch,heads", [(1, 1), (3, 2)])
def test_select_matches_reference(gpu, length, batch, heads):
    gen = torch.Generator(device="cuda").manual_seed(length)
    score = (torch.randn(batch, heads, length, generator=gen, device="cuda") * 2).exp()
    for budget in sorted({1, max(1, length // 3), max(1, length - 1), length, length + 7}):
        for first, last in {(0, 0), (min(4, budget), 0), (min(2, budget), min(budget - min(2, budget), 9)), (0, budget)}:
            _select_check(gpu, score, budget, first, last)


@pytest.mark.parametrize("length", [50, 3000, 70000])
def test_select_ties_and_special_scores(gpu, length):
    gen = torch.Generator(device="cuda").manual_seed(length)
    few = torch.randint(0, 3, (2, 2, length), generator=gen, device="cuda").float()
    few[0, 0] = 1.0                                            # all equal
    few[0, 1] = torch.where(few[0, 1] > 1, 0.0, -0.0)          # one value, two signs
    odd = torch.randn(2, 2, length, generator=gen, device="cuda")
    odd[0, 0, ::3] = float("nan")
    odd[0, 1, ::2] = float("-inf")
    odd[1, 0, ::5] = float("inf")
    odd[1, 1] = float("nan")
    odd[1, 0, 1] = torch.finfo(torch.float32).min
    tiny = torch.rand(2, 2, length, generator=gen, device="cuda") * 1e-40  # subnormal
    for score in (few, odd, tiny):
        for budget in (1, length // 3, length - 2):
            _select_check(gpu, score, budget)
            if budget > 8:
                _select_check(gpu, score, budget, 3, 4)


def test_select_ragged_lengths(gpu):
    s = 5000
    score = torch.randn(8, 3, s, device="cuda")
    lengths = torch.tensor([0, 1, 299, 300, 301, s, s + 9, -4], dtype=torch.int32, device="cuda")
    score[2, :, 299:] = float("inf")  # past the length: not read
    score[4, :, 301:] = float("nan")
    _select_check(gpu, score, 300, 4, 16, lengths)
    _select_check(gpu, score, 300, 300, 0, lengths)
    _select_check(gpu, score, 300, 0, 300, lengths)


def test_select_long_row_and_strides(gpu):
    score = torch.randn(1, 1, 1_000_003, device="cuda")
    _select_check(gpu, score, 65536, 4, 128)
    wide = torch.randn(2, 6, 9001, device="cuda")
    view = wide[:, 1:4, 7:8008]
    assert torch.equal(_select_check(gpu, view, 1000, 1, 5), gpu.evict_select(view.contiguous(), 1000, 1, 5)[0])


@pytest.mark.parametrize("rows", [(1, 8, 40000), (40, 8, 9000), (2, 2, 200000), (40, 8, 1500), (25, 8, 4096), (3, 1, 16385)], ids=str)
def test_select_many_shapes_of_work(gpu, rows):
    """Few long rows, many short ones: whatever the work is split into."""
    score = torch.rand(rows, device="cuda") ** 8
    _select_check(gpu, score, rows[2] // 7, 4, 64)


# --------------------------------------------------------------------- gather --

def _gather_plain(keep, x):
    there = keep >= 0
    b, h, n = keep.shape
    at = keep.long().clamp(min=0).reshape(b, h, n, *[1] * (x.dim() - 3)).expand(b, h, n, *x.shape[3:])
    y = x.gather(2, at)
    return torch.where(there.reshape(b, h, n, *[1] * (x.dim() - 3)), y, torch.zeros_like(y))


@pytest.mark.parametrize("width", [1, 3, 8, 64, 80, 100, 128, 576])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.bfloat16, torch.float32, torch.int64])
def test_gather_matches_indexing(gpu, width, dtype):
    b, h, s, n = 2, 3, 413, 77
    x = torch.randint(0, 100, (b, h, s, width), device="cuda").to(dtype)
    y = torch.randint(0, 100, (b, h, s, width), device="cuda").to(dtype)
    keep = torch.sort(torch.stack([torch.randperm(s, device="cuda")[:n] for _ in range(b * h)]).view(b, h, n), 2).values.int()
    keep[1, 1, 50:] = -1
    keep[0, 2, 3] = s  # outside: zeros
    score = torch.rand(b, h, s, device="cuda")
    got = gpu.evict_gather(keep, (x, y, score))
    keep = torch.where(keep < s, keep, -1)
    for g, src in zip(got, (x, y, score)):
        assert torch.equal(g, _gather_plain(keep, src))


def test_gather_strides_and_given_outputs(gpu):
    b, h, s, d, n = 2, 4, 300, 24, 50
    kv = torch.randn(b, s, 2, h, d, device="cuda").half()  # entries outside heads, keys beside values
    keys, values = (kv[:, :, i].transpose(1, 2) for i in (0, 1))
    keep = torch.sort(torch.randint(0, s, (b, h, n), device="cuda"), 2).values.int()
    cache = torch.full((2, b, h, 64, d), 7.0, device="cuda").half()
    out = (cache[0][:, :, :n], cache[1][:, :, 3:3 + n])
    gpu.evict_gather(keep, (keys, values), out=out)
    assert torch.equal(out[0], _gather_plain(keep, keys.contiguous()))
    assert torch.equal(out[1], _gather_plain(keep, values.contiguous()))
    assert (cache[0][:, :, n:] == 7).all() and (cache[1][:, :, :3] == 7).all() and (cache[1][:, :, 3 + n:] == 7).all()
    odd = torch.randn(b, h, s, d + 1, device="cuda").half()[..., 1:]  # entries on odd addresses
    assert torch.equal(gpu.evict_gather(keep, (odd,))[0], _gather_plain(keep, odd.contiguous()))


def test_gather_offsets_past_32_bits(gpu):
    s, d = 40_000_000, 128
    x = torch.zeros(1, 1, s, d, dtype=torch.uint8, device="cuda")  # 5 GB
    at = torch.tensor([0, 17_000_000, 34_000_001, s - 1], device="cuda")
    x[0, 0, at] = torch.arange(1, 5, dtype=torch.uint8, device="cuda")[:, None]
    got, = gpu.evict_gather(at.int().view(1, 1, 4), (x,))
    assert got[0, 0, :, 0].tolist() == [1, 2, 3, 4] and got[0, 0, :, -1].tolist() == [1, 2, 3, 4]


def test_select_then_gather_on_another_stream(gpu):
    b, h, s, d = 2, 2, 3000, 64
    score, keys = torch.rand(b, h, s, device="cuda"), torch.randn(b, h, s, d, device="cuda")
    keep, _ = gpu.evict_select(score, 100, 2, 8)
    want, = gpu.evict_gather(keep, (keys,))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine = keys + 0
    k2, _ = gpu.evict_select(score, 100, 2, 8, stream=side)
    got, = gpu.evict_gather(k2, (mine,), stream=side)
    side.synchronize()
    assert torch.equal(k2, keep) and torch.equal(got, want)


@pytest.mark.parametrize("rows", [(1, 2), (3, 5), (40, 8)], ids=str)
@pytest.mark.parametrize("width,dtype", [(128, torch.bfloat16), (80, torch.float16), (64, torch.uint8), (3, torch.float32),
                                         (1, torch.uint8), (576, torch.float32)])
def test_gather_in_place(gpu, rows, width, dtype):
    """The first budget entries of the arrays themselves: what a copy would hold, and the rest as it was."""
    b, h = rows
    s, n = (900, 333) if b * h > 100 else (7001, 3000)
    gen = torch.Generator(device="cuda").manual_seed(width)
    cache = torch.randint(0, 100, (2, b, h, s + 3, width), generator=gen, device="cuda").to(dtype)
    keys, values = cache[0][:, :, :s], cache[1][:, :, 2:2 + s]
    score = torch.rand(b, h, s, generator=gen, device="cuda")
    lengths = torch.tensor([[s, n - 40, n + 1][i % 3] for i in range(b)], dtype=torch.int32, device="cuda")
    keep, _ = gpu.evict_select(score, n, 5, 17, lengths)
    want = [_gather_plain(keep, x) for x in (keys, values, score)]
    rest = [x[:, :, n:].clone() for x in (keys, values, score)]
    edge = cache[1][:, :, :2].clone(), cache[0][:, :, s:].clone()
    gpu.evict_gather(keep, (keys, values, score), out=tuple(x[:, :, :n] for x in (keys, values, score)))
    for x, w, r in zip((keys, values, score), want, rest):
        assert torch.equal(x[:, :, :n], w) and torch.equal(x[:, :, n:], r)
    assert torch.equal(cache[1][:, :, :2], edge[0]) and torch.equal(cache[0][:, :, s:], edge[1])


def test_gather_in_place_of_the_whole_cache(gpu):
    """Nothing moves, or everything by one."""
    x = torch.randn(2, 3, 5000, 64, device="cuda")
    was = x.clone()
    same = torch.arange(5000, dtype=torch.int32, device="cuda").expand(2, 3, 5000).contiguous()
    gpu.evict_gather(same, (x,), out=(x,))
    assert torch.equal(x, was)
    gpu.evict_gather(torch.where(same < 4999, same + 1, -1), (x,), out=(x,))
    assert torch.equal(x[:, :, :-1], was[:, :, 1:]) and not x[:, :, -1].any()
