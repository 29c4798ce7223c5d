"""README's example of a decoding step gives what its calls promise."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decoding_example(gpu):
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    ns = {"om": gpu, "torch": torch}
    code, = [b for b in blocks if "beam_select" in b]
    exec(compile(code, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    assert ns["scores"].shape == ns["parents"].shape == ns["tokens"].shape == (2, 4)
    assert torch.all(ns["scores"][:, 1:] <= ns["scores"][:, :-1]) and int(ns["tokens"].max()) < 50021
    assert torch.equal(ns["x"], (ns["table"][ns["tokens"].flatten().long()].float() * 16).bfloat16())
    count = torch.bincount(ns["tokens"].flatten(), minlength=50021)
    assert torch.equal(ns["grad_table"], (16.0 * count)[:, None].expand(50021, 256).bfloat16())
    assert ns["y"].shape == (8, 256) and ns["y"].isfinite().all()
