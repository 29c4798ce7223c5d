"""om_accumulate_weights over very many rows: the error does not grow with their number as one running sum's does.

Rows are summed in blocks of 128, the blocks one after the other, over at most 8 warps: with u = 2^-24, n rows are
within (128 + n / 128 + 8 + 2) u of their sum's size (the last two: decay * score and its addition).
The rows are one row read again and again (stride 0), n a power of two: n times a value is exact.
"""
import pytest
import torch

from selection_reference import DTYPES, U32, f64

pytestmark = pytest.mark.gpu


def _check(om, row, heads, queries, out=None, score=None):
    w = row.expand(1, heads, queries, row.shape[0])
    n = heads * queries
    got = f64(om.accumulate_weights(w, score, kv_heads=1, out=out))[0, 0]
    want = f64(row) * n + (0 if score is None else f64(score)[0, 0])
    assert (abs(got - want) <= (128 + n / 128 + 10) * U32 * abs(want)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("start", [0, 1, 3])
def test_many_queries(gpu, dtype, start):
    """A whole prompt's queries; rows on 16 bytes and on odd addresses."""
    gen = torch.Generator(device="cuda").manual_seed(start)
    row = torch.rand(1003 + start, generator=gen, device="cuda").to(DTYPES[dtype])[start:]
    _check(gpu, row, 2, 32768)
    _check(gpu, row, 1, 4096, score=torch.rand(1, 1, row.shape[0], device="cuda"))


@pytest.mark.parametrize("shift", [0, 1])
def test_many_queries_of_a_long_cache(gpu, shift):
    """Tiles enough for one warp each; outputs on 16 bytes (written by the lanes) and not."""
    row = torch.rand(700_000, device="cuda")
    out = torch.empty(1, 1, row.shape[0] + 4, device="cuda")[:, :, shift:shift + row.shape[0]]
    _check(gpu, row, 1, 16384, out=out)


def test_rows_on_changing_addresses(gpu):
    """Odd row lengths: neighbouring rows start at one of 8 offsets, and blocks end where a warp comes to the next
    (through a batch of both: 16 times at most)."""
    w = torch.rand(1, 2, 8192, 1001, device="cuda").half()
    got = f64(gpu.accumulate_weights(w, kv_heads=1))[0, 0]
    want = f64(w)[0].sum((0, 1))
    assert (abs(got - want) <= (128 + 16384 / 128 + 16 + 10) * U32 * want).all()
