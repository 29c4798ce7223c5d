"""om_evict_gather at the greatest budget, whose last tile ends at 2^31 - 1 entries."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_gather_to_the_greatest_budget(gpu):
    n = 2 ** 31 - 1  # 8.6 GB of indices, 2.1 GB of output
    keep = torch.full((1, 1, n), -1, dtype=torch.int32, device="cuda")
    keep[0, 0, -300:] = torch.arange(300, dtype=torch.int32, device="cuda")
    src = torch.arange(1, 301, device="cuda").remainder(255).add(1).to(torch.uint8).view(1, 1, 300, 1)
    room = torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda")  # past the end: has to stay
    out = room[:n].view(1, 1, n, 1)
    gpu.evict_gather(keep, (src,), out=(out,))
    assert torch.equal(room[n - 300:n], src.view(-1))
    assert (room[n:] == 7).all()
    step = 1 << 28
    assert not any(bool(room[i:min(i + step, n - 300)].any()) for i in range(0, n - 300, step))
