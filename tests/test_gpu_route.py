"""om_route_topk and om_route_topk_backward against 64-bit references.

Inputs whose choice would hang on the rounding of exp are drawn anew (the gap
between neighbours is then at least GAP, 40 times what 32 bits can lose on
scores of at most 1), so ids are compared exactly.

Tolerance of the weights, relative: the exponent's argument x - top carries
|x - top| * 2^-24 <= 24 half ulps for logits within +-12, exp itself 2 ulps,
twice (numerator and sum), the sum of 1024 terms in a tree over 32 lanes of 32
terms 36 and the quotient and the scale 2: 80 half ulps in all.
"""
import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import DTYPES, U32, f64

pytestmark = pytest.mark.gpu

WEIGHT_TOL = 80 * U32
GAP = 1e-5


def _close_calls(x, k, score, bias, groups, picks, best):
    c = ref.choices(x, score, bias)
    bad = np.zeros(len(x), bool)
    near = lambda v: ((v[:, :-1] != v[:, 1:]) & (v[:, :-1] - v[:, 1:] < GAP * (np.abs(v[:, :-1]) + (bias is not None)))).any(1)  # noqa: E731
    if groups > 1 and picks < groups:
        by = -np.sort(-c.reshape(len(x), groups, -1), 2)[:, :, :best]
        total = by.sum(2)
        rank = np.argsort(-total, 1, kind="stable")
        v = np.take_along_axis(total, rank, 1)[:, picks - 1:picks + 1]
        bad |= near(v)
        for t in range(len(x)):
            for g in rank[t, picks:]:
                size = x.shape[1] // groups
                c[t, g * size:(g + 1) * size] = -np.inf
    v = -np.sort(-c, 1)[:, :k + 1]
    return bad | near(np.where(np.isfinite(v), v, -1e9))


def _logits(seed, tokens, experts, dtype, k, score, bias, groups, picks, best):
    gen = torch.Generator().manual_seed(seed)
    new = lambda n: (torch.randn(n, experts, generator=gen) * 2).clamp(-12, 12).to(DTYPES[dtype])  # noqa: E731
    x = new(tokens)
    for _ in range(60):
        bad = _close_calls(f64(x), k, score, bias, groups, picks, best)
        if not bad.any():
            return x
        x[torch.from_numpy(bad)] = new(int(bad.sum()))
    raise AssertionError("no unambiguous input found")


def _check_route(om, x, k, score="softmax", bias=None, groups=1, picks=1, best=1, renorm=False, scale=1.0, view=None):
    b = None if bias is None else torch.from_numpy(bias).float().cuda()
    xs = x.cuda() if view is None else view
    ids, w = om.route_topk(xs, k, score=score, bias=b, groups=groups, group_picks=picks, group_best=best,
                           renorm=renorm, scale=scale)
    want_ids, want_w = ref.route(f64(x), k, score, None if b is None else f64(b), groups, picks, best, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    fine = ~np.isnan(want_w)
    assert np.all(np.abs(got - want_w)[fine] <= WEIGHT_TOL * np.abs(want_w)[fine] + 1e-37)
    return ids, w


SHAPES = [  # tokens, experts, k, groups, picks, best
    (1, 1, 1, 1, 1, 1), (1, 64, 6, 1, 1, 1), (3, 7, 7, 1, 1, 1), (5, 33, 4, 1, 1, 1), (70, 32, 2, 4, 2, 1),
    (9, 160, 8, 8, 3, 2), (33, 256, 8, 8, 4, 2), (4, 257, 5, 1, 1, 1), (6, 96, 32, 32, 16, 2), (3, 1024, 32, 16, 4, 2),
    (2, 513, 1, 1, 1, 1), (300, 48, 5, 3, 2, 2), (2, 12, 3, 12, 3, 2),
    (17, 128, 4, 2, 1, 1), (9, 192, 6, 4, 2, 2), (5, 1024, 8, 8, 2, 1), (40, 64, 3, 8, 5, 2), (6, 320, 7, 1, 1, 1),
    (11, 1000, 8, 1, 1, 1),
    (21, 72, 4, 4, 2, 2), (7, 200, 8, 2, 1, 2), (6, 96, 6, 16, 4, 2), (5, 256, 8, 32, 8, 1), (4, 640, 8, 8, 2, 2),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_matches_reference(gpu, shape, score, dtype):
    tokens, experts, k, groups, picks, best = shape
    rng = np.random.default_rng(experts + k)
    for biased in (False, True):
        bias = rng.normal(size=experts).astype(np.float32).astype(np.float64) * (0.1 if score == "sigmoid" else 0.01) if biased else None
        x = _logits(experts * 3 + biased, tokens, experts, dtype, k, score, bias, groups, picks, best)
        for renorm, scale in ((False, 1.0), (True, 2.5)):
            _check_route(gpu, x, k, score, bias, groups, picks, best, renorm, scale)


@pytest.mark.parametrize("experts", [5, 64, 130, 1000])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_ties_go_to_the_lower_index(gpu, experts, renorm):
    rng = np.random.default_rng(experts)
    x = torch.from_numpy(rng.integers(-2, 3, (50, experts))).float()
    x[7] = 0.0
    x[8] = torch.where(torch.arange(experts) % 2 == 0, 0.0, -0.0)  # one value, two signs
    for score in ("softmax", "sigmoid"):
        _check_route(gpu, x, min(experts, 8), score, renorm=renorm)
        _check_route(gpu, x.half(), min(experts, 8), score, renorm=renorm)
    bias = np.zeros(experts)
    _check_route(gpu, x, min(experts, 8), "sigmoid", bias=bias, renorm=renorm)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks(gpu, dtype, score):
    """Rows that leave nothing, one expert, fewer than k; masked groups; the type's lowest value; NaN."""
    e, k = 72, 6
    x = (torch.arange(e).float().repeat(9, 1) * 7 % 73 / 16).to(DTYPES[dtype])
    ninf = -float("inf")
    x[0] = ninf
    x[1] = ninf
    x[1, 40] = 0.5
    x[2, 5:] = ninf
    x[3, :36] = ninf
    x[4] = torch.finfo(DTYPES[dtype]).min  # low, but there
    x[5, 3] = float("nan")
    x[6] = float("nan")
    x[7, 11] = torch.finfo(DTYPES[dtype]).min
    for renorm in (False, True):
        for groups, picks, best in ((1, 1, 1), (6, 2, 2), (6, 1, 1)):
            _check_route(gpu, x, k, score, groups=groups, picks=picks, best=best, renorm=renorm)
    bias = np.zeros(e)
    bias[::3] = -np.inf
    bias[1] = np.nan
    keep = [0, 1, 2, 3, 7, 8]
    _check_route(gpu, x[keep], k, score, bias=bias, groups=4, picks=2, best=2, renorm=True)


def test_route_extreme_logits(gpu):
    """Renormalised weights where every score underflows, and where the scores saturate."""
    x = torch.tensor([[-300.0, -301.0, -299.5, -400.0], [300.0, 301.0, 299.0, 298.0], [-100.0, 100.0, 0.0, 50.0]])
    for score in ("softmax", "sigmoid"):
        _check_route(gpu, x, 3, score, renorm=True)
    ids, _ = gpu.route_topk(x.cuda(), 2, score="sigmoid")  # 300 and 301 both score 1: still in order
    assert ids.tolist() == [[2, 0], [1, 0], [1, 3]]
    inf = torch.tensor([[0.0, float("inf"), 1.0, -1.0]])
    ids, w = gpu.route_topk(inf.cuda(), 2, score="sigmoid")
    assert ids.tolist() == [[1, 2]] and w[0, 0] == 1.0


def test_route_strided_rows_and_no_tokens(gpu):
    for dtype in (torch.float32, torch.bfloat16):
        wide = (torch.arange(37 * 300).reshape(37, 300) * 37 % 2003 / 256.0).to(dtype).cuda()
        for lo, e in ((0, 64), (1, 64), (3, 129), (17, 256)):
            view = wide[:, lo:lo + e]
            _check_route(gpu, view.cpu(), 4, "sigmoid", view=view)
        one = wide[0].expand(5, 300)  # a row that every token shares
        _check_route(gpu, one.cpu(), 4, "softmax", view=one)
    ids, w = gpu.route_topk(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert gpu.route_topk_backward(torch.empty(0, 8, device="cuda"), ids, w).shape == (0, 8)


def test_route_on_another_stream(gpu):
    side = torch.cuda.Stream()
    x = torch.randn(4000, 128, device="cuda")
    want = gpu.route_topk(x, 4)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x * 1.0
    got = gpu.route_topk(y, 4, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


BACK = [(1, 1, 1), (3, 7, 3), (5, 33, 4), (40, 64, 6), (9, 160, 8), (33, 256, 8), (3, 1024, 32), (4, 513, 2), (65, 48, 1)]


def _grad_close(got, want, grad, scale, k):
    """Each formula adds at most k terms g*w with sum w <= 1, then multiplies twice: (k + 160) half ulps of
    max |g| in 32 bits (80 for a weight, see above), and one rounding to the type: what comes out lies between
    the roundings of the interval's two ends."""
    tol = np.abs(grad).max(1, keepdims=True) * scale * (k + 160) * U32
    ends = [f64(torch.from_numpy(v).to(got.dtype)) for v in (want - tol, want + tol)]
    return bool(np.all((ends[0] <= f64(got)) & (f64(got) <= ends[1])))


@pytest.mark.parametrize("shape", BACK, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_backward_matches_formula(gpu, shape, score, renorm, dtype):
    tokens, experts, k = shape
    gen = torch.Generator().manual_seed(experts + k)
    x = (torch.randn(tokens, experts, generator=gen) * 2).clamp(-12, 12).to(DTYPES[dtype])
    ids = x.float().topk(k, 1).indices.to(torch.int32)
    if k > 1:
        ids[0, 1] = -1
        ids[-1, 0] = experts
    grad = torch.randn(tokens, k, generator=gen)
    got = gpu.route_topk_backward(x.cuda(), ids.cuda(), grad.cuda(), score=score, renorm=renorm, scale=2.5)
    assert got.dtype == x.dtype
    want = ref.route_backward(f64(x), ids.numpy(), f64(grad), score, renorm, 2.5)
    assert _grad_close(got, want, f64(grad), 2.5, k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_matches_differences(gpu, score, renorm):
    """Central differences of the forward call's own weights.  Step h = 2^-6; logits are 0.1 apart, so no
    choice changes.  Third derivatives of these weights are at most 1: truncation h^2 / 6 < 4.1e-5 for each of
    the k terms, rounding 80 half ulps of a weight <= 1 over h: 3.1e-4 each."""
    tokens, experts, k, h = 4, 24, 5, 2.0 ** -6
    gen = torch.Generator().manual_seed(1)
    x = torch.stack([torch.randperm(experts, generator=gen) for _ in range(tokens)]).float().cuda() * 0.1
    grad = torch.randn(tokens, k, generator=gen).cuda()
    ids, _ = gpu.route_topk(x, k, score=score, renorm=renorm)
    got = gpu.route_topk_backward(x, ids, grad, score=score, renorm=renorm)
    for e in range(experts):
        step = torch.zeros_like(x)
        step[:, e] = h
        up, dn = (gpu.route_topk(x + s, k, score=score, renorm=renorm) for s in (step, -step))
        assert torch.equal(up[0], ids) and torch.equal(dn[0], ids)
        slope = (((up[1] - dn[1]).double() / (2 * h)) * grad).sum(1)
        tol = grad.abs().sum(1) * (h * h / 6 + 80 * U32 / h)
        assert bool(((got[:, e] - slope).abs() <= tol).all())


def test_route_backward_masked_rows(gpu):
    x = torch.zeros(3, 8)
    x[0] = -float("inf")
    x[1, 2:] = -float("inf")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = gpu.route_topk(x.cuda(), 4, score=score, renorm=renorm)
            g = gpu.route_topk_backward(x.cuda(), ids, torch.ones_like(w), score=score, renorm=renorm)
            want = ref.route_backward(f64(x), ids.cpu().numpy(), np.ones((3, 4)), score, renorm)
            assert np.allclose(f64(g), want, rtol=0, atol=200 * U32)
            assert not g[0].any() and not g[1, 2:].any()


def test_route_backward_strided_logits(gpu):
    wide = torch.randn(19, 200, device="cuda")
    view = wide[:, 5:5 + 131]
    ids, w = gpu.route_topk(view, 6)
    g = torch.randn_like(w)
    assert torch.equal(gpu.route_topk_backward(view, ids, g), gpu.route_topk_backward(view.contiguous(), ids, g))


# ------------------------------------------- enough tokens for fewer lanes each --

MANY = 2600  # above the number up to which a token gets most lanes


def _route_all(x, k, score, bias, groups, picks, best, renorm, scale):
    """The reference for many rows at once: no masks, no NaN."""
    s = ref.scores(x, score)
    by_logit = bias is None and (groups == 1 or best == 1)
    c = x.copy() if by_logit else s + (0.0 if bias is None else bias)
    rows = np.arange(len(x))[:, None]
    if groups > 1:
        total = -np.sort(-c.reshape(len(x), groups, -1), 2)[:, :, :best].sum(2)
        out = np.argsort(-total, 1, kind="stable")[:, picks:]
        c.reshape(len(x), groups, -1)[rows, out] = -np.inf
    ids = np.argsort(-c, 1, kind="stable")[:, :k]
    w = s[rows, ids]
    return ids, (w / w.sum(1, keepdims=True) if renorm else w) * scale


@pytest.mark.parametrize("shape", [(64, 6, 1, 1, 1), (128, 8, 1, 1, 1), (160, 8, 8, 3, 2), (256, 8, 8, 4, 2), (256, 8, 8, 4, 1),
                                   (256, 5, 2, 1, 2), (257, 3, 1, 1, 1), (512, 8, 4, 2, 2), (72, 8, 4, 3, 2), (40, 1, 1, 1, 1),
                                   (96, 12, 1, 1, 1), (96, 6, 16, 4, 2), (256, 8, 32, 8, 1), (200, 8, 4, 2, 2), (90, 5, 3, 2, 2),
                                   (160, 16, 1, 1, 1), (256, 12, 8, 4, 2), (512, 9, 4, 3, 1), (67, 13, 1, 1, 1), (16, 16, 2, 2, 1)],
                         ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_many_tokens(gpu, shape, score, dtype):
    experts, k, groups, picks, best = shape
    rng = np.random.default_rng(experts + k)
    for biased in (False, True):
        bias = rng.normal(size=experts).astype(np.float32).astype(np.float64) * (0.1 if score == "sigmoid" else 0.01) if biased else None
        x = _logits(experts * 7 + biased, MANY, experts, dtype, k, score, bias, groups, picks, best)
        b = None if bias is None else torch.from_numpy(bias).float().cuda()
        for renorm in (False, True):
            ids, w = gpu.route_topk(x.cuda(), k, score=score, bias=b, groups=groups, group_picks=picks, group_best=best,
                                    renorm=renorm, scale=1.5)
            want_ids, want_w = _route_all(f64(x), k, score, None if b is None else f64(b), groups, picks, best, renorm, 1.5)
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            assert np.all(np.abs(f64(w) - want_w) <= WEIGHT_TOL * np.abs(want_w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,groups,picks", [(64, 1, 1), (130, 1, 1), (256, 8, 3)])
@pytest.mark.parametrize("k", [8, 15])
def test_route_many_tokens_ties_and_masks(gpu, dtype, experts, groups, picks, k):
    """A few values only, so most choices tie; some rows and experts masked."""
    rng = np.random.default_rng(experts)
    x = torch.from_numpy(rng.integers(-2, 2, (MANY, experts))).to(DTYPES[dtype])
    x[::7, ::3] = -float("inf")
    x[5::11, 1] = float("nan")
    x[13] = -float("inf")
    x[MANY - 1, 3:] = -float("inf")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(experts, device="cuda")):
            ids, w = gpu.route_topk(x.cuda(), k, score=score, bias=bias, groups=groups, group_picks=picks, renorm=True)
            rows = [*range(0, MANY, 97), 5, 13, 16, MANY - 1]
            want_ids, want_w = ref.route(f64(x[rows]), k, score, None if bias is None else f64(bias), groups, picks, 1, True)
            assert np.array_equal(ids.cpu().numpy()[rows], want_ids)
            assert np.all(np.abs(f64(w)[rows] - want_w) <= WEIGHT_TOL * want_w)


@pytest.mark.parametrize("experts,k", [(64, 6), (160, 8), (257, 3), (1000, 8), (48, 1), (96, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_backward_many_tokens(gpu, experts, k, score, renorm, dtype):
    gen = torch.Generator().manual_seed(experts + k)
    x = (torch.randn(MANY, experts, generator=gen) * 2).clamp(-12, 12).to(DTYPES[dtype])
    x[3, 2:] = -float("inf")
    x[4] = -float("inf")
    x[5, ::5] = float("nan")
    ids = torch.where(x.isnan(), torch.finfo(torch.float32).min, x.float()).topk(k, 1).indices.to(torch.int32)
    ids[MANY - 1, 0] = -1
    grad = torch.randn(MANY, k, generator=gen)
    got = gpu.route_topk_backward(x.cuda(), ids.cuda(), grad.cuda(), score=score, renorm=renorm, scale=2.5)
    rows = [0, 1, 3, 4, 5, *range(60, MANY, 101), MANY - 1]
    clean = torch.where(x.isnan(), -float("inf"), x.float())[rows]
    want = ref.route_backward(f64(clean), ids.numpy()[rows], f64(grad)[rows], score, renorm, 2.5)
    assert _grad_close(got[rows], want, f64(grad)[rows], 2.5, k)
