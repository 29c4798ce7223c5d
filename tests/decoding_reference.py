"""Plain implementations in 64 bits of the calls around the ordered selections, and the bounds of their errors."""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
E32 = 2.0 ** -24


def beam_scores(logits, scores=None, finished=None, end_id=0):
    """Every continuation's score [batch, beams, vocab] in 64 bits, -inf where there is none."""
    x = logits.double()
    x = torch.where(x.isnan(), -torch.inf, x)
    lse = torch.logsumexp(x, 2, keepdim=True)
    p = torch.zeros(logits.shape[:2], dtype=torch.float64, device=x.device) if scores is None else scores.double()
    c = torch.where(x > -torch.inf, p[:, :, None] + (x - lse), -torch.inf)
    c = torch.where(c.isnan(), -torch.inf, c)
    if finished is not None:
        c[finished] = -torch.inf
        c[:, :, end_id] = torch.where(finished, torch.where(p.isnan(), -torch.inf, p), c[:, :, end_id])
    return c


def beam_tolerance(logits, c):
    """Error of a score: its own rounding, and the logarithm's: terms whose argument x - max is rounded twice, of
    weight in the sum only up to log(vocab) + 20 below the maximum (2 * 33 half steps), 2 steps of the exponential,
    and sums of at most vocab / 1024 terms a thread, then 5 + 4 + 16 levels."""
    return E32 * (66 + 8 + logits.shape[2] / 1024 + 40) + E32 * c.abs()


def check_beams(got, logits, top, scores=None, finished=None, end_id=0):
    """A choice is right if every chosen continuation has its score, those of one beam are its greatest logits
    (ties to the lower token), and none left out is greater than a chosen one by more than the scores' error."""
    out, parents, tokens = (t.cpu() for t in got)
    logits = logits.cpu()
    scores = None if scores is None else scores.cpu()
    finished = None if finished is None else finished.cpu()
    c = beam_scores(logits, scores, finished, end_id)
    batch, beams, vocab = c.shape
    assert out.shape == parents.shape == tokens.shape == (batch, top)
    for b in range(batch):
        flat = c[b].flatten()
        n = min(top, int((flat > -torch.inf).sum()))
        assert torch.all(parents[b, n:] == -1) and torch.all(tokens[b, n:] == -1) and torch.all(out[b, n:] == -torch.inf)
        if n == 0:
            continue
        p, t = parents[b, :n].long(), tokens[b, :n].long()
        assert (0 <= int(p.min()) and int(p.max()) < beams and 0 <= int(t.min()) and int(t.max()) < vocab)
        want = c[b, p, t]
        tol = beam_tolerance(logits, want)
        assert torch.all(want > -torch.inf)
        assert torch.all((out[b, :n].double() - want).abs() <= tol)
        assert torch.all(out[b, 1:n] <= out[b, :n - 1])  # greatest first, as given
        for i in range(beams):
            mine = t[p == i]
            order = c[b, i].sort(descending=True, stable=True).indices
            assert torch.equal(mine, order[:len(mine)])
        left = flat.clone()
        left[p * vocab + t] = -torch.inf
        assert n == len(set((p * vocab + t).tolist()))
        assert float(left.max()) <= float(want.min() + 2 * tol.max())


def embed_backward(grad, ids, rows, scale=1.0, base=None):
    """(gradient of the table, error bound of its sum in 32 bits): pieces of 32 or 128 terms, then the pieces."""
    g, i = grad.double().flatten(0, -2), ids.flatten().long()
    there = (i >= 0) & (i < rows)
    g, i = g[there], i[there]
    total = torch.zeros(rows, g.shape[-1], dtype=torch.float64, device=g.device)
    total.index_add_(0, i, g)
    size = torch.zeros_like(total).index_add_(0, i, g.abs())
    count = torch.bincount(i, minlength=rows).double()[:, None]
    total, size = total * scale, size * abs(scale)
    error = E32 * (count.clamp(max=128) + count / 32 + 3) * size
    if base is not None:
        total = total + base.double()
        error = error + E32 * total.abs()
    return total, error


ACT = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}


def expert_mlp(x, ids, weights, up, down, gate=None, act="silu"):
    """(y, error bound).  A product of k columns in 32 bits: k / 16 sums of the matrix instruction, each within a step
    of what it adds, and 16 more; the activations' slopes are at most 1.2 and their values within 4 steps; they go on
    as two values (twice half a step of the type, down to f16's smallest step 2^-24 of the second)."""
    x, up, down, w = x.double(), up.double(), down.double(), weights.double()
    tokens, hidden = x.shape
    inner = up.shape[1]
    half = HALF[torch.bfloat16] if DT[0] == torch.bfloat16 else HALF[torch.float16]
    e1, e2 = (hidden / 16 + 16) * 2 * E32, (inner / 16 + 16 + ids.shape[1]) * 2 * E32
    y = torch.zeros(tokens, hidden, dtype=torch.float64, device=x.device)
    error = torch.zeros_like(y)
    f = ACT[act]
    for t in range(tokens):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < up.shape[0]:
                continue
            u, du = up[e] @ x[t], e1 * (up[e].abs() @ x[t].abs())
            if gate is not None:
                g, dg = gate[e].double() @ x[t], e1 * (gate[e].double().abs() @ x[t].abs())
                h = f(g) * u
                dh = 1.2 * dg * (u.abs() + du) + (f(g).abs() + 8 * E32 * (1 + g.abs())) * du + 8 * E32 * (f(g).abs() + g.abs()) * u.abs()
            else:
                h = f(u)
                dh = 1.2 * du + 8 * E32 * (h.abs() + u.abs())
            dh = dh + half * half * h.abs() + 2.0 ** -25
            y[t] += w[t, j] * (down[e] @ h)
            error[t] += w[t, j].abs() * (down[e].abs() @ (dh + e2 * h.abs()))
    return y, error


DT = [torch.bfloat16]  # the type that expert_mlp bounds (set by its tests)
