"""The bounds of the decoding tests notice planted mistakes (on the CPU)."""
import torch

import decoding_reference as ref


def test_reference_sees_a_lost_column():
    """The bound of these tests against a planted mistake: one column of the second product left out (on the CPU)."""
    gen = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, up, down = rand(2, 64).bfloat16(), (rand(2, 1100, 64) / 8).bfloat16(), (rand(2, 64, 1100) / 33).bfloat16()
    ids, w = torch.tensor([[0], [1]], dtype=torch.int32), torch.ones(2, 1)
    ref.DT[0] = torch.bfloat16
    want, error = ref.expert_mlp(x, ids, w, up, down)
    down[:, :, 1030] = 0
    got, _ = ref.expert_mlp(x, ids, w, up, down)
    bound = error + ref.HALF[torch.bfloat16] * (want.abs() + error) + 2.0 ** -25
    assert float(((got - want).abs() > bound).float().mean()) > 0.2
