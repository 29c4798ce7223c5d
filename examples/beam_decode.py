"""Beam search over a small model with routed experts, and the training of its embedding.

    python examples/beam_decode.py

One decoding step as the library's calls make it up, for all beams of a batch:

  tokens    their rows of the embedding, scaled (embed_lookup)
  attention over the beams' caches, plain torch
  experts   chosen by a router (route_topk) and multiplied in one launch (expert_mlp)
  beams     the best continuations of every sequence (beam_select); the caches of the
            beams that go on move to their new places (beam_gather), but for the
            entries of the prompt, which all beams of a sequence share

and the embedding's training: the rows that a batch asks for carry their gradient to the
table (embed_lookup's backward pass, which sums equal tokens in their order).
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ordered_merge_gb300 as om  # noqa: E402


class Model:
    """A decoder layer between an embedding and its transpose; bfloat16."""

    def __init__(self, vocab=1000, hidden=128, heads=4, experts=16, inner=64, picks=4, device="cuda"):
        new = lambda *s: (torch.randn(*s, device=device) * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.vocab, self.hidden, self.heads, self.picks = vocab, hidden, heads, picks
        self.table = new(vocab, hidden)
        self.q, self.k, self.v, self.o = (new(hidden, hidden) for _ in range(4))
        self.router = new(experts, hidden)
        self.gate_up, self.down = new(experts, 2 * inner, hidden), new(experts, hidden, inner)
        self.gate, self.up = self.gate_up[:, :inner], self.gate_up[:, inner:]

    def caches(self, batch, beams, capacity):
        width = self.hidden // self.heads
        return [torch.zeros(batch, beams, self.heads, capacity, width, device=self.table.device, dtype=self.table.dtype)
                for _ in range(2)]

    def step(self, tokens, caches, used):
        """Logits [batch, beams, vocab] of the tokens [batch, beams]; their keys and values go to place `used`."""
        batch, beams = tokens.shape
        x = om.embed_lookup(tokens.contiguous(), self.table, scale=math.sqrt(self.hidden))
        split = lambda y: y.view(batch, beams, self.heads, 1, -1)  # noqa: E731
        keys, values = (c[:, :, :, :used + 1] for c in caches)
        keys[:, :, :, used:], values[:, :, :, used:] = split(x @ self.k.t()), split(x @ self.v.t())
        weights = (split(x @ self.q.t()) @ keys.transpose(3, 4)).float().div_(math.sqrt(keys.shape[4])).softmax(4)
        x = x + (weights.to(x.dtype) @ values).flatten(2) @ self.o.t()
        rows = x.flatten(0, 1)
        ids, weights = om.route_topk(rows @ self.router.t(), self.picks, renorm=True)
        rows = rows + om.expert_mlp(rows, ids, weights, self.up, self.down, gate=self.gate)
        rows = rows * rows.float().square().mean(1, keepdim=True).add(1e-6).rsqrt().to(rows.dtype)
        return (rows @ self.table.t()).view(batch, beams, self.vocab)


def beam_search(model, prompts, beams, steps, end_id):
    """The `beams` best continuations of each prompt [batch, n]: (tokens [batch, beams, steps], scores)."""
    batch, n = prompts.shape
    one = model.caches(batch, 1, n + steps)  # the prompt, once for all beams of a sequence
    for i in range(n):
        logits = model.step(prompts[:, i:i + 1], one, i)
    scores, parents, tokens = om.beam_select(logits, beams)
    caches = [c.expand(-1, beams, -1, -1, -1).contiguous() for c in one]
    history = tokens[:, :, None]
    finished = tokens == end_id
    starts = torch.full((batch,), n, device=prompts.device, dtype=torch.int32)
    for i in range(1, steps):
        logits = model.step(tokens, caches, n + i - 1)
        scores, parents, tokens = om.beam_select(logits, beams, scores, finished=finished, end_id=end_id)
        om.beam_gather(parents, caches, starts=starts, lengths=starts + i)  # in place, the prompt left alone
        at = parents.long()
        finished = finished.gather(1, at) | (tokens == end_id)
        history = torch.cat([history.gather(1, at[:, :, None].expand(-1, -1, i)), tokens[:, :, None]], 2)
    return history, scores


def next_token_loss(table, out, tokens):
    """Cross entropy of each token's successor, from its own row of the table alone."""
    rows = om.embed_lookup(tokens[:, :-1].contiguous(), table)
    return torch.nn.functional.cross_entropy((rows @ out).flatten(0, 1), tokens[:, 1:].flatten())


def main():
    torch.manual_seed(0)
    model = Model()
    prompts = torch.randint(3, model.vocab, (3, 5), device="cuda")
    tokens, scores = beam_search(model, prompts, beams=4, steps=12, end_id=2)
    for b in range(len(prompts)):
        print(f"prompt {b}: best {tokens[b, 0].tolist()} at {scores[b, 0].item():.3f}, last beam at {scores[b, -1].item():.3f}")

    # a table learns which token follows which
    follows = torch.randperm(200, device="cuda")
    table = (0.1 * torch.randn(200, 64, device="cuda")).requires_grad_()
    out = torch.randn(64, 200, device="cuda") / 8
    for step in range(41):
        tokens = torch.randint(0, 200, (16, 1), device="cuda")
        for _ in range(15):
            tokens = torch.cat([tokens, follows[tokens[:, -1:]]], 1)
        loss = next_token_loss(table, out, tokens)
        grad, = torch.autograd.grad(loss, table)
        with torch.no_grad():
            table -= 20.0 * grad
        if step % 20 == 0:
            print(f"step {step}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
