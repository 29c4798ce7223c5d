"""om_embed_lookup and its gradient against their definitions in 64 bits."""
import pytest
import torch

import decoding_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 2, 3, 8, 63, 64, 100, 258, 1024, 4100])
def test_lookup(gpu, dtype, width):
    gen = _gen(width)
    table = torch.randn(301, width, generator=gen, device="cuda").to(dtype)
    for n, ids_type, scale in ((1, torch.int64, 1.0), (7, torch.int32, 0.5), (1000, torch.int64, width ** 0.5)):
        ids = torch.randint(0, 301, (n,), generator=gen, device="cuda").to(ids_type)
        got = gpu.embed_lookup(ids, table, scale)
        want = table[ids.long()]
        assert torch.equal(got, (want.float() * scale).to(dtype))
        exact = want.double() * torch.tensor(scale, dtype=torch.float32).double().item()
        # a product rounded to 32 bits and then to the type
        assert torch.all((got.double() - exact).abs() <= (ref.HALF[dtype] + 2 * ref.E32) * exact.abs() + 2.0 ** -25)


def test_lookup_ids_outside_and_shapes(gpu):
    table = torch.randn(10, 48, device="cuda")
    ids = torch.tensor([[3, -1, 9], [10, 0, -2 ** 63]], device="cuda")
    got = gpu.embed_lookup(ids, table)
    assert got.shape == (2, 3, 48)
    want = torch.where(((ids >= 0) & (ids < 10))[..., None], table[ids.clamp(0, 9)], 0.0)
    assert torch.equal(got, want)
    assert torch.equal(gpu.embed_lookup(torch.tensor([2 ** 31 - 1, 9], dtype=torch.int32, device="cuda"), table)[0], torch.zeros(48, device="cuda"))
    big = torch.tensor([2 ** 32 + 3], device="cuda")  # not row 3
    assert not gpu.embed_lookup(big, table).any()
    assert gpu.embed_lookup(torch.zeros(0, dtype=torch.int64, device="cuda"), table).shape == (0, 48)
    assert not gpu.embed_lookup(ids, table[:0]).any()
    nan = table.clone()
    nan[5] = float("nan")
    assert not gpu.embed_lookup(ids, nan).isnan().any()


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_strided_tables(gpu, dtype):
    for shift in range(9):
        buf = torch.randn(40 * 72 + 16, device="cuda").to(dtype)
        table = buf[shift:shift + 40 * 72].view(40, 72)[:, :64]
        ids = torch.randint(0, 40, (77,), device="cuda")
        assert torch.equal(gpu.embed_lookup(ids, table), table[ids])
        out = torch.zeros(77 * 64 + 16, device="cuda", dtype=dtype)[shift:shift + 77 * 64].view(77, 64)
        assert gpu.embed_lookup(ids, table, out=out) is out
        assert torch.equal(out, table[ids])


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_odd_rows_and_guards(gpu, dtype):
    ids = torch.tensor([3, -1, 0, 6, 6, 2, 7, 5], device="cuda")
    for width in (*range(1, 20), 31, 33, 127, 1025):
        for shift in range(9):
            apart = width + shift % 3
            buf = torch.randn(7 * apart + 16, device="cuda").to(dtype)
            table = buf[8 - shift:8 - shift + 7 * apart].view(7, apart)[:, :width]
            around = torch.full((8 * width + 32,), 99.0, device="cuda", dtype=dtype)
            out = around[shift:shift + 8 * width].view(8, width)
            gpu.embed_lookup(ids, table, 2.0, out=out)
            want = torch.where(((ids >= 0) & (ids < 7))[:, None], table[ids.clamp(0, 6)] * 2, 0.0)
            assert torch.equal(out, want)  # doubling rounds nothing
            assert torch.all(around[:shift] == 99) and torch.all(around[shift + 8 * width:] == 99)


def test_lookup_offsets_past_32_bits(gpu):
    table = torch.zeros(1 << 20, 2200, dtype=torch.float16, device="cuda")  # 4.6 GB
    table[-1], table[(1 << 20) - 7, -1] = 3.0, 4.0
    got = gpu.embed_lookup(torch.tensor([(1 << 20) - 1, 0, (1 << 20) - 7], device="cuda"), table)
    assert torch.all(got[0] == 3) and not got[1].any() and got[2, -1] == 4 and not got[2, :-1].any()


# ------------------------------------------------------------- gradient --

def _check_backward(om, grad, ids, rows, scale=1.0, into=None, base=None, table=None):
    """The gradient of a table of `rows` rows, written or (base) added, in type `into`."""
    out_type = into or grad.dtype
    if table is None:
        table = torch.full((rows, grad.shape[-1]), 777.0, device="cuda", dtype=out_type)
    if base is not None:
        table.copy_(base)
    got = om.embed_lookup_backward(grad, ids, rows, scale, accumulate=base is not None, grad_table=table)
    assert got is table
    want, error = ref.embed_backward(grad, ids, rows, torch.tensor(scale).double().item(), base)
    bound = error + ref.HALF[out_type] * (want.abs() + error) + (2.0 ** -25 if out_type == torch.float16 else 2.0 ** -133)
    assert torch.all((got.double() - want).abs() <= bound)
    return got


IDS = {
    "spread": lambda n, rows, gen: torch.randint(0, rows, (n,), generator=gen, device="cuda"),
    "skewed": lambda n, rows, gen: (torch.rand(n, generator=gen, device="cuda") ** 8 * rows).long(),
    "one": lambda n, rows, gen: torch.full((n,), rows // 2, device="cuda"),
    "outside": lambda n, rows, gen: torch.randint(-rows, 2 * rows, (n,), generator=gen, device="cuda"),
    "none": lambda n, rows, gen: torch.full((n,), -1, device="cuda"),
    "ends": lambda n, rows, gen: torch.randint(0, 2, (n,), generator=gen, device="cuda") * (rows - 1),
}


@pytest.mark.parametrize("kind", list(IDS))
@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 128, 129, 1000, 5000])
def test_backward_runs(gpu, kind, n):
    gen = _gen(n)
    for rows, width, dtype in ((1, 40, torch.float32), (50, 64, torch.bfloat16), (3001, 33, torch.float16), (200, 1100, torch.float32)):
        grad = torch.randn(n, width, generator=gen, device="cuda").to(dtype)
        _check_backward(gpu, grad, IDS[kind](n, rows, gen), rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 2, 5, 8, 31, 32, 36, 260, 1023, 1024, 1025, 2052, 5000])
def test_backward_widths(gpu, dtype, width):
    gen = _gen(width)
    grad = torch.randn(700, width, generator=gen, device="cuda").to(dtype)
    for ids_type in (torch.int32, torch.int64):
        ids = IDS["skewed"](700, 90, gen).to(ids_type)
        _check_backward(gpu, grad, ids, 90, 3.0)
        _check_backward(gpu, grad, ids, 90, 0.25, into=torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("into_f32", [False, True])
def test_backward_accumulates(gpu, dtype, into_f32):
    gen = _gen(5)
    into = torch.float32 if into_f32 else dtype
    for n in (0, 40, 3000):
        grad = torch.randn(n, 130, generator=gen, device="cuda").to(dtype)
        base = torch.randn(77, 130, generator=gen, device="cuda").to(into)
        _check_backward(gpu, grad, IDS["skewed"](n, 77, gen), 77, 2.0, into, base)


def test_backward_many_tokens(gpu):
    gen = _gen(9)
    n, rows, width = 300_007, 40_000, 24
    grad = torch.randn(n, width, generator=gen, device="cuda")
    for kind in ("spread", "skewed", "one"):
        _check_backward(gpu, grad, IDS[kind](n, rows, gen), rows)


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 16385, 40_000, 262_144, 262_145])
def test_backward_ways_of_sorting(gpu, n):
    """Tokens up to which they are counted, sorted by one cluster, and merged; short and long pieces."""
    gen = _gen(n)
    for rows, width in ((3000, 16), (1, 8), (600_000, 4)):
        grad = torch.randn(n, width, generator=gen, device="cuda")
        for kind in ("skewed", "one", "outside"):
            _check_backward(gpu, grad, IDS[kind](n, rows, gen), rows)
    # a run that ends, and one that starts, at every place around a piece's end
    lengths = torch.arange(1, 2 * int((2 * n) ** 0.5), device="cuda")
    ids = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), lengths)[:n]
    ids = ids[torch.randperm(len(ids), generator=gen, device="cuda")].contiguous()
    _check_backward(gpu, torch.randn(len(ids), 8, generator=gen, device="cuda"), ids, len(lengths))


def test_backward_strided_table_and_guards(gpu):
    gen = _gen(11)
    for shift in range(5):
        grad = torch.randn(300, 20, generator=gen, device="cuda").bfloat16()
        buf = torch.full((60 * 24 + 16,), 5.0, device="cuda").bfloat16()
        table = buf[shift:shift + 60 * 24].view(60, 24)[:, :20]
        _check_backward(gpu, grad, IDS["outside"](300, 60, gen), 60, table=table)
        table.fill_(5.0)
        assert torch.all(buf == 5.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_backward_odd_rows(gpu, dtype):
    gen = _gen(12)
    for width, n in ((7, 20000), (257, 900), (1031, 300)):
        for shift in range(9):
            flat = torch.randn(n * width + 16, generator=gen, device="cuda").to(dtype)
            flat[:shift], flat[shift + n * width:] = float("nan"), float("nan")  # none of the rows' values
            grad = flat[shift:shift + n * width].view(n, width)
            into = torch.float32 if shift % 2 else dtype
            buf = torch.full((90 * (width + 2) + 16,), 5.0, device="cuda", dtype=into)
            table = buf[8 - shift:8 - shift + 90 * (width + 2)].view(90, width + 2)[:, 1:width + 1]
            base = torch.randn(90, width, generator=gen, device="cuda").to(into) if shift % 3 == 0 else None
            _check_backward(gpu, grad, IDS["skewed"](n, 90, gen), 90, 0.5, into, base, table)
            table.fill_(5.0)
            assert torch.all(buf == 5.0)


def test_backward_repeats_bit_for_bit_and_on_a_stream(gpu):
    gen = _gen(12)
    grad = torch.randn(20_000, 96, generator=gen, device="cuda").bfloat16()
    ids = IDS["skewed"](20_000, 500, gen)
    want = gpu.embed_lookup_backward(grad, ids, 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = gpu.embed_lookup_backward(grad, ids, 500, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_autograd(gpu):
    """Gradient through autograd against the formula's (64 bits) and against differences."""
    gen = _gen(13)
    table = torch.randn(40, 12, generator=gen, device="cuda").requires_grad_()
    ids = torch.randint(-2, 42, (5, 9), generator=gen, device="cuda")
    pull = torch.randn(5, 9, 12, generator=gen, device="cuda")
    y = gpu.embed_lookup(ids, table, 1.5)
    (y * pull).sum().backward()
    want, error = ref.embed_backward(pull, ids, 40, 1.5)
    assert torch.all((table.grad.double() - want).abs() <= error + ref.E32 * want.abs() * 2)
    # the lookup is linear: a difference is exact but for the rounding of its two ends
    with torch.no_grad():
        for _ in range(3):
            step = torch.randn(40, 12, generator=gen, device="cuda")
            ends = [(gpu.embed_lookup(ids, table + s * step, 1.5).double() * pull).sum() for s in (0.5, -0.5)]
            slope = (table.grad.double() * step).sum()
            scale = (gpu.embed_lookup(ids, table.abs() + step.abs(), 1.5).double() * pull.abs()).sum() + (want.abs() * step.abs()).sum()
            assert abs(ends[0] - ends[1] - slope) <= 16 * ref.E32 * scale
    # a gradient that is one value for all (sum().backward()), and a second backward that adds
    table.grad = None
    gpu.embed_lookup(ids, table).sum().backward()
    gpu.embed_lookup(ids.int(), table).sum().backward()
    count = torch.bincount(ids[(ids >= 0) & (ids < 40)], minlength=40)
    assert torch.equal(table.grad, 2.0 * count[:, None].expand(40, 12))
    assert not gpu.embed_lookup(ids, table.detach()).requires_grad
    with torch.no_grad():
        assert not gpu.embed_lookup(ids, table).requires_grad
