"""The example's layer against dense torch: the experts' sum and the router's gradient, the bounded cache's
contents, and the calls captured in a CUDA graph as a decoding loop replays them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(request):
    spec = importlib.util.spec_from_file_location("decoder_step", os.path.join(ROOT, "examples", "decoder_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_experts_match_dense_products(gpu, example, score, renorm):
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    t, d, e, k = 37, 16, 12, 3
    x, router, up, down = rand(t, d), rand(d, e), rand(e, d, 8) / 4, rand(e, 8, d) / 4
    r32 = router.float().requires_grad_()
    y, load = example.experts_forward(x.float(), r32, up.float(), down.float(), k, score=score, renorm=renorm)
    r64 = router.clone().requires_grad_()
    logits = x @ r64
    s = logits.softmax(1) if score == "softmax" else logits.sigmoid()
    w, ids = s.topk(k, 1)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    each = torch.nn.functional.silu(torch.einsum("td,edh->teh", x, up))
    dense = torch.einsum("teh,ehd->ted", each, down)
    want = (dense.gather(1, ids[:, :, None].expand(-1, -1, d)) * w[:, :, None]).sum(1)
    assert load.tolist() == torch.bincount(ids.reshape(-1), minlength=e).tolist()
    # 32-bit products of 16 terms, twice, and sums of k: well below 1e-4 of the largest value
    assert (y - want).abs().max() <= 1e-4 * want.abs().max()
    pull = rand(t, d)
    g32, = torch.autograd.grad((y * pull.float()).sum(), r32)
    g64, = torch.autograd.grad((want * pull).sum(), r64)
    assert (g32 - g64).abs().max() <= 1e-4 * g64.abs().max()


def test_cache_is_cut_to_its_budget(gpu, example):
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache = example.BoundedCache(2, 2, 40, 8, budget=20, first=2, last=5, dtype=torch.float32)
    shadow = [[[] for _ in range(2)] for _ in range(2)]  # (key, score) of the entries that stay
    for step in range(60):
        k, v = (torch.randn(2, 2, 1, 8, generator=gen, device="cuda") for _ in range(2))
        full = cache.used + 1 > 40
        cache.append(k, v)
        q = torch.randn(2, 4, 1, 8, generator=gen, device="cuda")
        for b in range(2):
            for h in range(2):
                rows = shadow[b][h]
                if full:
                    n = len(rows)
                    middle = sorted(range(2, n - 5), key=lambda i: (-rows[i][1], i))[:20 - 2 - 5]
                    rows[:] = [rows[i] for i in [0, 1, *sorted(middle), *range(n - 5, n)]]
                rows.append([k[b, h, 0], 0.0])
        cache.attend(q)
        score = cache.score.tolist()
        for b in range(2):
            for h in range(2):
                assert len(shadow[b][h]) == cache.used == int(cache.lengths[b])
                for i, row in enumerate(shadow[b][h]):
                    assert score[b][h][i] >= row[1]  # weights only add
                    row[1] = score[b][h][i]
                assert torch.equal(torch.stack([r[0] for r in shadow[b][h]]), cache.keys[b, h, :cache.used])


def test_example_runs(gpu, example, capsys):
    example.main()
    lines = capsys.readouterr().out.splitlines()
    losses = [float(line.split("loss ")[1].split(",")[0]) for line in lines if "loss" in line]
    assert losses[-1] < losses[0]


def test_calls_in_a_cuda_graph(gpu):
    """A decoding step's selections captured once and replayed on new inputs."""
    logits = torch.randn(64, 128, device="cuda")
    ids_all = torch.randint(-1, 128, (200_000,), dtype=torch.int32, device="cuda")
    w = torch.rand(2, 8, 1, 5000, device="cuda")
    score = torch.zeros(2, 2, 5000, device="cuda")
    keys = torch.randn(2, 2, 5000, 64, device="cuda")

    def step():
        ids, weights = gpu.route_topk(logits, 4)
        grad = gpu.route_topk_backward(logits, ids, weights)
        groups = gpu.group_by_id(ids, 128)
        many = gpu.group_by_id(ids_all, 128)
        total = gpu.accumulate_weights(w, score)
        keep, kept = gpu.evict_select(total, 700, 4, 32)
        return (ids, weights, grad, *groups, *many, total, keep, kept, *gpu.evict_gather(keep, (keys, total)))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        torch.manual_seed(seed)
        logits.normal_(), w.uniform_(), keys.normal_()
        ids_all.random_(-1, 128)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, step()):
            assert torch.equal(got, want)
