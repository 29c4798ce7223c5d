"""om_route_topk_backward of a plain softmax, entry by entry.

With half ulps u = 2^-24, logits whose differences are exact in 32 bits, S = sum |g w| over the picks:
exp has 2 ulps (4 u), the row's sum 32 terms a lane and 5 levels (37 u), so 1 / sum 42 u and a weight 47 u;
dot = sum g w has 47 u, a rounding of scale * g, one of the product and 5 levels: 54 u of S.
An expert not picked, s_e * dot: 54 + 43 (dot / sum) + 5 (its term): 102 u of s_e * S.
A pick, w * (g - dot): 52 u of w * |g| and 105 u of w * S.
Terms and results below the normal range have 2^-149 apart: at most 2 such steps of a term, times dot / sum,
and one of the result.
"""
import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import DTYPES, U32, f64

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8, 2), (5, 33, 4), (40, 64, 6), (9, 160, 8), (33, 256, 8), (3, 1024, 32), (4, 513, 2), (3000, 160, 8),
          (2600, 64, 1), (2600, 257, 3), (2600, 1000, 8)]


def _case(tokens, experts, k, dtype):
    """Logits in 16ths, most of them near the top and every fifth far below it; positive gradients, so that the
    picks' sum does not cancel."""
    gen = torch.Generator().manual_seed(experts + k)
    x = torch.randint(-64, 65, (tokens, experts), generator=gen) / 16.0
    x[:, ::5] -= torch.randint(0, 90, (tokens, len(range(0, experts, 5))), generator=gen)
    x = x.to(DTYPES[dtype])
    ids = x.float().topk(k, 1).indices.to(torch.int32)
    grad = torch.rand(tokens, k, generator=gen) + 0.5
    return x, ids, grad


def _bounds(x, ids, grad, scale):
    """The gradient in 64 bits and how far 32 bits may be from it."""
    s = ref.scores(f64(x), "softmax")
    at, rows = ids.numpy().astype(np.int64), np.arange(len(s))[:, None]
    g = np.zeros_like(s)
    g[rows, at] = f64(grad) * scale
    dot = (g * s).sum(1, keepdims=True)
    want = s * (g - dot)
    picked = np.zeros_like(s)
    picked[rows, at] = 1
    top = f64(x).max(1, keepdims=True)
    total = np.exp(f64(x) - top).sum(1, keepdims=True)
    tol = s * U32 * np.where(picked == 1, 52 * np.abs(g) + 105 * dot, 102 * dot) + (2 * dot / total + 1) * 2.0 ** -149
    return want, tol


def _within(got, want, tol):
    """Between the roundings to got's type of the interval's ends."""
    ends = [f64(torch.from_numpy(v).to(got.dtype)) for v in (want - tol, want + tol)]
    return (ends[0] <= f64(got)) & (f64(got) <= ends[1])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_every_entry_of_a_softmax_gradient(gpu, shape, dtype):
    tokens, experts, k = shape
    x, ids, grad = _case(tokens, experts, k, dtype)
    got = gpu.route_topk_backward(x.cuda(), ids.cuda(), grad.cuda(), scale=2.5)
    want, tol = _bounds(x, ids, grad, 2.5)
    assert _within(got, want, tol).all()
    # nothing here passes for zero: not where the type can hold it
    there = np.abs(want) > (0 if dtype == "f32" else 1e-4 if dtype == "f16" else 1e-30)
    there &= np.abs(want) > 2.0 ** -145
    assert there.any() and not _within(torch.zeros_like(x), want, tol)[there].any()
