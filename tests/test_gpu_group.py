"""om_group_by_id against a stable argsort, and against the library's own key+value sort."""
import numpy as np
import pytest
import torch

import selection_reference as ref

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 31, 32, 33, 511, 1000, 4095, 8192, 8193, 20000, 100003, 1 << 20]


def _check(om, ids, groups):
    got = om.group_by_id(torch.from_numpy(ids).cuda(), groups)
    for g, w in zip(got, ref.group(ids, groups)):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("groups", [1, 2, 8, 255, 256, 1024])
def test_group_matches_stable_sort(gpu, n, groups):
    rng = np.random.default_rng(n + groups)
    _check(gpu, rng.integers(0, groups, n).astype(np.int32), groups)
    skew = (rng.random(n) ** 6 * groups).astype(np.int32)
    skew[rng.random(n) < 0.1] = -1
    _check(gpu, skew, groups)


@pytest.mark.parametrize("n", [40, 30000])
def test_group_ids_outside(gpu, n):
    """Ids below, at and far past the groups are one last group, in slot order."""
    ids = np.tile(np.array([3, -1, 0, 4, np.iinfo(np.int32).max, 1, np.iinfo(np.int32).min, 3], np.int32), n // 8)
    _check(gpu, ids, 4)
    _check(gpu, np.full(n, -7, np.int32), 4)   # nothing inside
    _check(gpu, np.full(n, 2, np.int32), 4)    # one group has all


def test_group_is_the_librarys_stable_sort(gpu):
    ids = torch.randint(0, 64, (50021,), dtype=torch.int32, device="cuda")
    _, order, _ = gpu.group_by_id(ids, 64)
    keys, slots = ids.clone(), torch.arange(ids.numel(), dtype=torch.int32, device="cuda")
    gpu.merge_sort_u32(keys, slots)
    assert torch.equal(order, slots)


def test_group_shapes_streams_and_repeats(gpu):
    ids = torch.randint(-1, 16, (999, 8), dtype=torch.int32, device="cuda")
    want = gpu.group_by_id(ids, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine = ids + 0
    got = [gpu.group_by_id(mine, 16, stream=side) for _ in range(3)]
    side.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    big = torch.randint(-1, 300, (300007,), dtype=torch.int32, device="cuda")
    first = gpu.group_by_id(big, 300)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(gpu.group_by_id(big, 300), first))
