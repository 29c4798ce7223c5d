"""Arrays that lie between each other's rows without sharing a byte: keys and values of one buffer, scores and
outputs of one buffer."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _layout(name, b, h, n, d):
    """Keys and values [b, h, n, d] of one buffer."""
    if name == "beside":      # batch, 2, heads, entries
        kv = torch.randn(b, 2, h, n, d, device="cuda")
        return kv[:, 0], kv[:, 1]
    if name == "heads":       # batch, heads, 2, entries
        kv = torch.randn(b, h, 2, n, d, device="cuda")
        return kv[:, :, 0], kv[:, :, 1]
    if name == "entries":     # batch, entries, 2, heads
        kv = torch.randn(b, n, 2, h, d, device="cuda")
        return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    kv = torch.randn(b, h, n, 2 * d, device="cuda")  # an entry's key, then its value
    return kv[..., :d], kv[..., d:]


LAYOUTS = ["beside", "heads", "entries", "widths"]


def _plain(keep, x):
    at = keep.long().clamp(min=0)[..., None].expand(*keep.shape, x.shape[3])
    return torch.where(keep[..., None] >= 0, x.gather(2, at), 0.0)


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("b,h", [(1, 1), (3, 2), (1, 4), (4, 1)])
def test_gather_into_one_buffer(gpu, name, b, h):
    n, d, budget = 90, 16, 33
    keys, values = _layout(name, b, h, n, d)
    keep, _ = gpu.evict_select(torch.rand(b, h, n, device="cuda"), budget)
    out = _layout(name, b, h, budget, d)
    gpu.evict_gather(keep, (keys, values), out=out)
    assert torch.equal(out[0], _plain(keep, keys)) and torch.equal(out[1], _plain(keep, values))


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("b,h", [(1, 1), (3, 2), (1, 4), (4, 1)])
def test_gather_in_place_in_one_buffer(gpu, name, b, h):
    n, d, budget = 900, 16, 333
    keys, values = _layout(name, b, h, n, d)
    keep, _ = gpu.evict_select(torch.rand(b, h, n, device="cuda"), budget)
    want = [torch.cat([_plain(keep, x), x[:, :, budget:]], 2) for x in (keys, values)]
    gpu.evict_gather(keep, (keys, values), out=(keys[:, :, :budget], values[:, :, :budget]))
    assert torch.equal(keys, want[0]) and torch.equal(values, want[1])


def test_accumulate_beside_the_old_scores(gpu):
    w = torch.rand(3, 4, 2, 50, device="cuda")
    both = torch.rand(3, 2, 2, 50, device="cuda")
    want = gpu.accumulate_weights(w, both[:, 0].contiguous(), decay=0.5)
    got = gpu.accumulate_weights(w, both[:, 0], decay=0.5, out=both[:, 1])
    assert torch.equal(got, want)
    wide = torch.rand(3, 2, 100, device="cuda")
    want = gpu.accumulate_weights(w, wide[..., :50].contiguous(), decay=0.5)
    assert torch.equal(gpu.accumulate_weights(w, wide[..., :50], decay=0.5, out=wide[..., 50:]), want)


def test_bytes_that_are_shared_are_refused(gpu):
    b, h, n, d = 2, 2, 40, 16
    kv = torch.zeros(b, 2, h, n, d, device="cuda")
    keys, values = kv[:, 0], kv[:, 1]
    keep = torch.zeros(b, h, 8, dtype=torch.int32, device="cuda")
    rows = torch.zeros(b, 2 * n, h, d, device="cuda").transpose(1, 2)
    other = torch.zeros(b, h, 20, d, device="cuda")
    wide = torch.zeros(b, h, n, 2 * d, device="cuda")
    for arrays, out in (
        ((keys,), (keys[:, :, 4:12],)),                             # into itself, shifted
        ((keys, values), (values[:, :, :8], keys[:, :, :8])),       # into each other
        ((rows[:, :, :n],), (rows[:, :, n - 1:n + 7],)),            # one entry
        ((keys, values), (other[:, :, :8], other[:, :, 7:15])),     # one entry of the outputs
        ((wide[..., :9],), (wide[:, :, :8, 8:17],)),                # one element of an entry
    ):
        with pytest.raises(gpu.OrdMergeError):
            gpu.evict_gather(keep, arrays, out=out)
    w = torch.rand(b, h, 1, 20, device="cuda")
    row = torch.zeros(b, h, 40, device="cuda")
    with pytest.raises(gpu.OrdMergeError):
        gpu.accumulate_weights(w, row[..., :20], out=row[..., 19:39])
