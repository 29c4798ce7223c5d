"""One decoder layer that routes its tokens to experts and keeps a bounded cache.

    python examples/decoder_step.py

The ordered selections as a model uses them together:

  cache     attention weights are summed into a score per entry
            (accumulate_weights); when the cache is full it is cut to its budget
            by them (evict_select) and moved (evict_gather)
  experts   a router scores the experts of each token (route_topk), the slots
            are grouped by expert (group_by_id), each expert multiplies its own
            rows, and the rows come back weighted; the router learns through the
            weights' gradient, and a bias evens out the experts' loads

Attention and the experts' products are plain torch: only their order is the
library's business here.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ordered_merge_gb300 as om  # noqa: E402


class BoundedCache:
    """Keys and values [batch, heads, capacity, width] with a score per entry."""

    def __init__(self, batch, heads, capacity, width, budget, first=4, last=16, device="cuda", dtype=torch.bfloat16):
        self.keys = torch.zeros(batch, heads, capacity, width, device=device, dtype=dtype)
        self.values = torch.zeros_like(self.keys)
        self.score = torch.zeros(batch, heads, capacity, device=device)
        self.lengths = torch.zeros(batch, device=device, dtype=torch.int32)
        self.used = 0  # the greatest length, on the host
        self.budget, self.first, self.last = budget, first, last

    def append(self, keys, values):
        """Adds [batch, heads, n, width] entries, cutting the cache first where they would not fit."""
        n = keys.shape[2]
        if self.used + n > self.keys.shape[2]:
            self.evict()
        at = slice(self.used, self.used + n)
        self.keys[:, :, at], self.values[:, :, at], self.score[:, :, at] = keys, values, 0.0
        self.lengths += n
        self.used += n

    def attend(self, q):
        """Softmax attention of q [batch, q_heads, n, width] over the entries; its weights are added to the score."""
        batch, q_heads, n, width = q.shape
        heads = self.keys.shape[1]
        keys = self.keys[:, :, :self.used].repeat_interleave(q_heads // heads, 1)
        values = self.values[:, :, :self.used].repeat_interleave(q_heads // heads, 1)
        logits = (q @ keys.transpose(2, 3)).float() / math.sqrt(width)
        # the n queries are the last n entries: each sees those up to its own
        ahead = torch.arange(self.used, device=q.device) > torch.arange(self.used - n, self.used, device=q.device)[:, None]
        weights = logits.masked_fill(ahead, -math.inf).softmax(3).to(q.dtype)
        score = self.score[:, :, :self.used]
        om.accumulate_weights(weights, score, lengths=self.lengths, out=score)
        return weights @ values

    def evict(self):
        score = self.score[:, :, :self.used]
        keep, kept = om.evict_select(score, self.budget, self.first, self.last, self.lengths)
        arrays = [x[:, :, :self.used] for x in (self.keys, self.values, self.score)]
        self.used = min(self.used, self.budget)
        om.evict_gather(keep, arrays, out=[x[:, :, :self.budget] for x in (self.keys, self.values, self.score)])
        self.lengths = kept


def experts_forward(x, router, up, down, top_k, bias=None, **options):
    """sum over the picks of weight * down[e] @ silu(up[e] @ x) for the rows of x, and the experts' loads."""
    experts = router.shape[1]
    ids, weights = om.route_topk(x @ router, top_k, bias=bias, **options)
    offsets, order, place = om.group_by_id(ids, experts)
    rows = x[(order // top_k).long()]  # grouped by expert
    ends = offsets.tolist()
    out = [torch.nn.functional.silu(rows[ends[e]:ends[e + 1]] @ up[e]) @ down[e] for e in range(experts)]
    out.append(rows.new_zeros(len(rows) - ends[-1], x.shape[1]))  # slots without an expert
    back = torch.cat(out)[place.long()].view(len(x), top_k, -1)
    return (back * weights[:, :, None].to(x.dtype)).sum(1), offsets.diff()


def main():
    torch.manual_seed(0)
    batch, q_heads, heads, width, hidden, experts, top_k = 2, 8, 2, 64, 128, 32, 4
    new = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16) / math.sqrt(s[-2] if len(s) > 1 else 1)  # noqa: E731
    router, up, down = new(hidden, experts), new(experts, hidden, 4 * hidden // top_k), new(experts, 4 * hidden // top_k, hidden)
    bias = torch.zeros(experts, device="cuda")
    options = dict(score="sigmoid", groups=4, group_picks=2, group_best=2, renorm=True)

    cache = BoundedCache(batch, heads, 256, width, budget=128)
    for step in range(200):  # a prompt of 64, then one token at a time
        n = 64 if step == 0 else 1
        cache.append(new(batch, heads, n, width) * 8, new(batch, heads, n, width))
        attended = cache.attend(new(batch, q_heads, n, width) * 8)
        x = attended.mean(1).reshape(batch * n, width).repeat(1, hidden // width)
        experts_forward(x, router, up, down, top_k, bias, **options)
    print("cache:", cache.used, "entries of", 263, "appended; lengths", cache.lengths.tolist())

    # the router alone learns to route like another one; the bias evens out the loads
    x, up, down = torch.randn(2048, hidden, device="cuda"), up.float(), down.float()
    router, teacher = router.float().requires_grad_(), router.float() + 0.5 * new(hidden, experts).float()
    options = dict(score="softmax", renorm=True)
    with torch.no_grad():
        want, _ = experts_forward(x, teacher, up, down, top_k, **options)
    optimizer = torch.optim.Adam([router], lr=2e-3)
    for step in range(61):
        y, load = experts_forward(x, router, up, down, top_k, bias, **options)
        loss = ((y - want) ** 2).mean() / (want ** 2).mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        bias -= 1e-4 * (load.float() - load.float().mean()).sign()
        if step % 20 == 0:
            print(f"step {step}: loss {loss.item():.4f}, busiest expert {int(load.max())} of {2048 * top_k} slots")


if __name__ == "__main__":
    main()
