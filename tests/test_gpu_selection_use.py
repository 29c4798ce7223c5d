"""The ordered selections as programs meet them: refusals by their messages, masks with many tokens, choices one
unit in the last place apart, several streams and threads, tensors past 2^31 elements, the README's examples."""
import os
import re
import threading

import numpy as np
import pytest
import torch

import selection_reference as ref
from selection_reference import DTYPES, U32, f64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MANY = 2600  # tokens that get the fewest lanes each


# ------------------------------------------------------------------ refusals --

def _refusals(om):
    x = torch.zeros(4, 8, device="cuda")
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    a = torch.zeros(1, 2, 3, 4, device="cuda")
    s = torch.zeros(1, 2, 9, device="cuda")
    keep = torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda")
    keys = torch.zeros(1, 2, 9, 4, device="cuda")
    return {
        "float32, bfloat16 or float16": lambda: om.route_topk(x.double(), 2),
        "logits must have 2 dimensions": lambda: om.route_topk(x[0], 2),
        "last dimension of logits": lambda: om.route_topk(x.t(), 2),
        "'softmax' or 'sigmoid'": lambda: om.route_topk(x, 2, score="relu"),
        "bias must be": lambda: om.route_topk(x, 2, bias=torch.zeros(7, device="cuda")),
        "bias must be a CUDA tensor": lambda: om.route_topk(x, 2, bias=torch.zeros(8)),
        "ids must be .*int32": lambda: om.route_topk(x, 2, ids=w),
        "weights must be .*float32": lambda: om.route_topk(x, 2, weights=w[:, :1]),
        "ids must have 2 dimensions": lambda: om.route_topk_backward(x, ids[0], w),
        "grad_weights must be": lambda: om.route_topk_backward(x, ids, w.double()),
        "grad_logits must be": lambda: om.route_topk_backward(x, ids, w, grad_logits=x.half()),
        "contiguous int32": lambda: om.group_by_id(w, 8),
        "offsets must be": lambda: om.group_by_id(ids, 8, offsets=ids),
        "kv_heads is needed": lambda: om.accumulate_weights(a),
        "score must be float32 of shape": lambda: om.accumulate_weights(a, s),
        "out must be float32 of shape": lambda: om.accumulate_weights(a, kv_heads=2, out=s),
        "lengths must be": lambda: om.accumulate_weights(a, kv_heads=2, lengths=torch.zeros(1, device="cuda")),
        "score must be float32 ": lambda: om.evict_select(s.half(), 2),
        "kept must be": lambda: om.evict_select(s, 2, kept=torch.zeros(2, dtype=torch.int32, device="cuda")),
        "no arrays": lambda: om.evict_gather(keep, ()),
        "keep must be": lambda: om.evict_gather(keep.long(), (keys,)),
        "out must hold one tensor": lambda: om.evict_gather(keep, (keys,), out=()),
        "out must be torch.float32": lambda: om.evict_gather(keep, (keys,), out=(a.half(),)),
        "out must have shape": lambda: om.evict_gather(keep, (keys,), out=(a[..., :3],)),
        "as many entries each": lambda: om.evict_gather(keep, (keys, keys[:, :, :8])),
        "entries of array must be contiguous": lambda: om.evict_gather(keep, (keys[..., ::2],)),
        "with batch 1 and heads 2": lambda: om.evict_gather(keep, (keys[:, :1],)),
    }


def test_refusals_by_their_messages(gpu):
    for message, call in _refusals(gpu).items():
        with pytest.raises(ValueError, match=message):
            call()
    for call in (lambda: gpu.route_topk(torch.zeros(4, 8, device="cuda"), 9),
                 lambda: gpu.route_topk(torch.zeros(4, 8, device="cuda"), 2, groups=3),
                 lambda: gpu.evict_select(torch.zeros(1, 2, 9, device="cuda"), 4, first=3, last=2)):
        with pytest.raises(gpu.OrdMergeError, match="OM_EINVAL"):
            call()


# ---------------------------------------------------------- masks and closeness --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,k", [(64, 8, 6), (256, 8, 8), (96, 4, 12), (160, 1, 16)])
def test_masks_with_many_tokens(gpu, dtype, score, experts, groups, k):
    """-inf and NaN biases and logits, whole groups and rows masked, two greatest to a group."""
    gen = torch.Generator().manual_seed(experts)
    # values a 64th apart and biases a 1024th: no two choices hang on a rounding, many are equal
    x = (torch.randint(-6, 7, (MANY, experts), generator=gen) / 2).to(DTYPES[dtype])
    size = experts // groups
    x[::3, :size] = -float("inf")
    x[1::5, ::4] = float("nan")
    x[2::7, 1:] = -float("inf")
    x[11] = -float("inf")
    bias = np.zeros(experts)
    bias[::6] = -np.inf
    bias[1::9] = np.nan
    if groups > 1:
        bias[2 * size:3 * size] = -np.inf
    rows = [*range(0, MANY, 53), 1, 2, 11, 16, MANY - 1]
    picks = max(1, groups // 2)
    b = torch.from_numpy(bias).float().cuda()
    ids, w = gpu.route_topk(x.cuda(), k, score=score, bias=b, groups=groups, group_picks=picks,
                            group_best=2 if groups > 1 else 1, renorm=True)
    few, _ = gpu.route_topk(x[rows].cuda(), k, score=score, bias=b, groups=groups, group_picks=picks,
                            group_best=2 if groups > 1 else 1, renorm=True)
    assert torch.equal(ids[rows], few)
    want, want_w = ref.route(f64(x[rows]), k, score, bias, groups, picks, 2 if groups > 1 else 1, True)
    assert np.array_equal(ids.cpu().numpy()[rows], want)
    # as for the weights elsewhere: 80 half ulps
    assert np.all(np.abs(f64(w)[rows] - want_w) <= 80 * U32 * want_w)


@pytest.mark.parametrize("tokens", [3, MANY])
@pytest.mark.parametrize("k", [4, 12, 20])
def test_logits_one_unit_apart(gpu, tokens, k):
    """With no bias the order is the logits' own, however close; with one, that of score + bias in 32 bits."""
    gen = torch.Generator().manual_seed(k)
    order = torch.stack([torch.randperm(96, generator=gen) for _ in range(tokens)])
    x = (1.5 + order * 2.0 ** -23).cuda()  # neighbours in float32
    want = order.argsort(1, descending=True)[:, :k]
    for score in ("softmax", "sigmoid"):
        for groups in (1, 4):
            ids, _ = gpu.route_topk(x, k, score=score, groups=groups, group_picks=groups)
            assert torch.equal(ids.cpu().long(), want)
    bias = (torch.randperm(96, generator=gen) * 2.0 ** -23).cuda()  # 0.5 + bias is exact
    ids, _ = gpu.route_topk(torch.zeros(tokens, 96, device="cuda"), k, score="sigmoid", bias=bias)
    assert (ids.cpu().long() == bias.cpu().argsort(descending=True)[:k]).all()


# ------------------------------------------------------------ streams and threads --

def _work(om, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    logits = rand(3000, 128)
    ids, w = om.route_topk(logits, 8, renorm=True)
    some = om.group_by_id(ids, 128)
    many = om.group_by_id((rand(400_000) * 130).int() - 1, 128)
    score = rand(2, 2, 60_000)
    keep, kept = om.evict_select(score, 20_000, 4, 64)
    cache = rand(2, 2, 60_000, 16)
    copy, = om.evict_gather(keep, (cache,))
    om.evict_gather(keep, (cache,), out=(cache[:, :, :20_000],))
    total = om.accumulate_weights(rand(2, 8, 3, 5001), kv_heads=2)
    back = om.route_topk_backward(logits, ids, w)
    return ids, w, *some, *many, keep, kept, copy, cache, total, back


def test_two_streams_and_two_threads(gpu):
    want = [_work(gpu, seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    for _ in range(5):
        streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]

        def run(i):
            with torch.cuda.stream(streams[i]):
                got[i] = _work(gpu, i + 1)

        threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for mine, theirs in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(mine, theirs))


def test_inputs_written_just_before(gpu):
    """The inputs come from kernels that still run when the call is launched, again and again into the same memory."""
    x = torch.empty(20_000, 128, device="cuda")
    score = torch.empty(4, 4, 30_000, device="cuda")
    slow = torch.randn(4096, 4096, device="cuda")
    for seed in range(8):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new_x, new_s = torch.randn(x.shape, generator=gen, device="cuda"), torch.rand(score.shape, generator=gen, device="cuda")
        torch.cuda.synchronize()
        torch.mm(slow, slow)
        x.copy_(new_x)
        ids, w = gpu.route_topk(x, 6)
        groups = gpu.group_by_id(ids, 128)
        score.copy_(new_s)
        keep, _ = gpu.evict_select(score, 3000)
        cut, = gpu.evict_gather(keep, (score,))
        x.zero_(), score.zero_()  # and are gone right after
        want, want_w = gpu.route_topk(new_x, 6)
        torch.cuda.synchronize()
        assert torch.equal(ids, want) and torch.equal(w, want_w)
        assert np.array_equal(groups[1].cpu().numpy(), ref.group(ids.cpu().numpy(), 128)[1])
        assert torch.equal(keep.long(), new_s.sort(dim=2, descending=True, stable=True).indices[..., :3000].sort().values)
        assert torch.equal(cut, new_s.gather(2, keep.long()))


# ------------------------------------------------------------------ large tensors --

def test_logits_past_31_bits(gpu):
    tokens, experts, k = 8_500_000, 256, 2  # 2.18e9 bf16 values
    x = torch.zeros(tokens, experts, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(tokens, device="cuda") * 7 % experts
    x.scatter_(1, at[:, None], 4.0)
    ids, w = gpu.route_topk(x, k)
    second = torch.where(at == 0, 1, 0)  # the others tie
    assert torch.equal(ids.long(), torch.stack([at, second], 1))
    grad = gpu.route_topk_backward(x, ids, torch.ones_like(w), score="sigmoid")
    assert torch.equal(grad[-1], grad[(tokens - 1) % 256]) and grad[-1].count_nonzero() == 2


def test_weights_past_31_bits(gpu):
    w = torch.zeros(1, 2, 1100, 1_000_001, dtype=torch.bfloat16, device="cuda")  # 2.2e9 values, rows on odd addresses
    w[0, :, ::100, -5:] = 1.0
    w[0, 1, -1, 3] = 2.0
    got = gpu.accumulate_weights(w, kv_heads=2)
    assert (got[0, :, -5:] == 11).all() and got[0, 1, 3] == 2 and got.sum() == 2 * 5 * 11 + 2


# ------------------------------------------------------------------------ README --

def test_every_readme_example_runs(gpu):
    """In their order, in one namespace; the ones for several GPUs need a process group and are left out."""
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), flags=re.S)
    ns = {}
    for code in blocks:
        if "distributed" not in code:
            exec(compile(code, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    ids, weights, keep = ns["ids"], ns["weights"], ns["keep"]
    assert ids.shape == weights.shape == (512, 8) and torch.allclose(weights.sum(1), torch.full((512,), 2.5, device="cuda"))
    assert torch.equal(ns["order"].long(), ids.view(-1).sort(stable=True).indices)
    assert torch.equal(ns["cache"][:, :, :256], ns["cut"])
    assert torch.equal(ns["cut_score"], ns["score"][:, :, :256]) and keep.shape == (2, 2, 256)
