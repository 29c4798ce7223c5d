"""Cases for measuring the ordered-selection operators of language models.

Four operators, each an ordering problem decided by a score with ties going to
the lowest index:

  route       scores of a router's logits, a balance bias, groups, the top k
              experts of every token and their weights; and its gradient
  group       the stable grouping of (token, pick) slots by expert
  weights     attention weights summed into a score per cache entry
  evict       the cache entries that stay (first ones, last ones, greatest
              scores), kept in order, and the cache gathered to them

`own` chooses between the plain forms below (elementary torch operations in 32
bits) and the library's calls.  listed() gives the fixed cases, draw() others
of the same ranges, exact() the operators' definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases --

def _route(name, tokens, experts, k, dtype, score, bias=False, groups=1, picks=1, best=1, renorm=False, scale=1.0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "picks": picks, "best": best, "renorm": renorm, "scale": scale}


def _route_back(name, tokens, experts, k, dtype, score, renorm=False, scale=1.0):
    return {"name": name, "op": "route_back", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype,
            "score": score, "renorm": renorm, "scale": scale}


def _group(name, slots, groups, dropped):
    return {"name": name, "op": "group", "slots": slots, "groups": groups, "dropped": dropped}


def _weights(name, batch, q_heads, kv_heads, queries, length, dtype, decay):
    return {"name": name, "op": "weights", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "queries": queries, "length": length, "dtype": dtype, "decay": decay}


def _evict(name, batch, heads, length, width, budget, first, last, dtype):
    return {"name": name, "op": "evict", "batch": batch, "heads": heads, "length": length, "width": width,
            "budget": budget, "first": first, "last": last, "dtype": dtype}


def listed():
    return [
        # one sequence decoding one token: the smallest call, all latency
        _route("route-one-token", 1, 64, 6, "bf16", "softmax"),
        # a training microbatch with a balance bias and limited groups, scores in 32 bits
        _route("route-biased-groups", 4096, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
        # a long prefill, an odd number of tokens
        _route("route-prefill", 131071, 128, 8, "bf16", "softmax", renorm=True),
        # the gradient of a renormalised sigmoid router on a microbatch of odd length
        _route_back("route-back-sigmoid", 4099, 256, 8, "f32", "sigmoid", True, 2.5),
        # the gradient of a softmax router over a large batch, a number of experts that is no power of two
        _route_back("route-back-softmax", 65536, 160, 6, "bf16", "softmax"),
        # the slots of 64 decoding sequences with 8 picks each
        _group("group-decode", 64 * 8, 256, False),
        # the slots of a microbatch, a few dropped for capacity
        _group("group-microbatch", 4096 * 8, 256, True),
        # the slots of a long prefill of odd length
        _group("group-prefill", 131071 * 8, 128, False),
        # one decoding step of a batch: one query, eight query heads to a cache head, ragged lengths
        _weights("weights-decode", 64, 64, 8, 1, 8192, "bf16", 0.99),
        # the last 32 queries of a long prompt whose length is odd, so rows start on odd addresses
        _weights("weights-window", 1, 32, 8, 32, 65539, "f16", 1.0),
        # one short conversation cut to its budget
        _evict("evict-short", 1, 8, 4096, 128, 1024, 4, 32, "bf16"),
        # a batch of long documents cut to an eighth
        _evict("evict-long", 4, 8, 131072, 128, 16384, 4, 512, "bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_back", "group", "weights", "evict", "evict"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("route", "route_back"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        experts = groups * rng.randint(max(1, 8 // groups), 256 // groups)
        k = rng.randint(1, min(8, experts))
        tokens = _spread(rng, 1, min(65536, 131071 * 128 // experts // SIZE[dtype]))
        score, renorm = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
        scale = rng.choice([1.0, 2.5])
        case = (_route if op == "route" else _route_back)("", tokens, experts, k, dtype, score)
        case.update(renorm=renorm, scale=scale)
        if op == "route":
            size = experts // groups
            picks = rng.randint(min(groups, -(-k // size)), groups)
            case.update(bias=rng.random() < 0.5, groups=groups, picks=picks, best=rng.choice([1, 2]))
    elif op == "group":
        case = _group("", _spread(rng, 1, 131071 * 8), rng.randint(2, 512), rng.random() < 0.5)
    elif op == "weights":
        kv_heads, share = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        queries = rng.choice([1, 1, _spread(rng, 2, 64)])
        most = 64 * 64 * 8192 * 2 // SIZE[dtype] // (kv_heads * (share + 4) * queries)
        length = _spread(rng, 16, min(131072, most))
        batch = _spread(rng, 1, max(1, min(64, most // length)))
        case = _weights("", batch, kv_heads * share, kv_heads, queries, length, dtype, rng.choice([1.0, 0.95]))
    else:
        batch, heads, width = _spread(rng, 1, 8), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128])
        length = _spread(rng, 64, min(131072, 131072 * 16 // (batch * heads)))
        budget = max(8, int(length * rng.uniform(0.05, 0.9)))
        most = 32 * 16384 * 128 * 2 // (batch * heads * width * SIZE[dtype])  # no more to move than the largest listed case
        budget = min(budget, most)
        first, last = rng.randint(0, 4), rng.randint(0, min(budget // 4, 512))
        case = _evict("", batch, heads, length, width, budget, first, last, dtype)
    case.pop("name")
    return case


def _lengths(case):
    """Valid entries of each sequence of a ragged batch; the first is full."""
    return [case["length"] - (b * 2654435761) % (case["length"] // 4 + 1) for b in range(case["batch"])]


def work(case):
    op = case["op"]
    if op in ("route", "route_back"):
        t, e, k, size = case["tokens"], case["experts"], case["k"], SIZE[case["dtype"]]
        if op == "route":  # logits in; ids and weights out
            return {"bytes": t * e * size + t * k * 8 + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
        # ids and the weights' gradients in, the logits' gradients out; only a softmax that is not
        # renormalised depends on more than the picked logits
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": t * e * size + (t * e if dense else t * k) * size + t * k * 8,
                "flops": 6 * t * e if dense else 8 * t * k}
    if op == "group":  # ids in; offsets, order and place out
        return {"bytes": case["slots"] * 12 + 4 * (case["groups"] + 1), "flops": 0}
    valid = sum(_lengths(case))
    if op == "weights":
        rows = case["q_heads"] * case["queries"]
        return {"bytes": valid * rows * SIZE[case["dtype"]] + valid * case["kv_heads"] * 4
                + case["batch"] * case["length"] * case["kv_heads"] * 4, "flops": valid * rows}
    kept = sum(min(n, case["budget"]) for n in _lengths(case))
    heads, slots = case["heads"], case["batch"] * case["budget"]
    entry = 2 * case["width"] * SIZE[case["dtype"]] + 4
    return {"bytes": heads * (valid * 4 + kept * entry + slots * (entry + 4)) + case["batch"] * 8, "flops": 0}


# ----------------------------------------------------------------- inputs --

def _unsure(case, logits, bias):
    """Rows whose decision hangs on the rounding of exp (in 64 bits: a gap below a few parts in
    a million, but not none).  Either answer is right there, so such rows are drawn anew."""
    x = logits.double()
    if case["score"] == "softmax":
        s = torch.softmax(x, 1)
    else:
        s = torch.sigmoid(x)
    c = s if bias is None else s + bias.double()
    near = lambda v, w, room: (v != w) & ((v - w).abs() < 4e-6 * (v.abs() + w.abs() + room))  # noqa: E731
    room = 0.0 if bias is None else float(s.max()) * (1.0 if case["score"] == "sigmoid" else 0.1)
    bad = torch.zeros(x.shape[0], dtype=torch.bool, device=x.device)
    g, picks = case["groups"], case["picks"]
    if g > 1 and picks < g:
        by = c.view(x.shape[0], g, -1)
        total = by.topk(min(case["best"], by.shape[2]), 2).values.sum(2)
        ranked, at = total.sort(dim=1, descending=True, stable=True)
        bad |= near(ranked[:, picks - 1], ranked[:, picks], room)
        keep = torch.zeros_like(total, dtype=torch.bool).scatter_(1, at[:, :picks], True)
        c = torch.where(keep[:, :, None], by, -math.inf).flatten(1)
    v = c.topk(min(case["k"] + 1, c.shape[1]), 1).values
    bad |= (near(v[:, :-1], v[:, 1:], room) & torch.isfinite(v[:, 1:])).any(1)
    return bad


def _logits(case, gen):
    t, e, dtype = case["tokens"], case["experts"], TYPES[case["dtype"]]
    popular = torch.randn(e, generator=gen, device="cuda") * 0.5  # some experts are asked for more often
    return popular, (torch.randn(t, e, generator=gen, device="cuda") * 1.5 + popular).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, new = case["op"], lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device="cuda")
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        popular, logits = _logits(case, gen)
        bias = None
        if case["bias"]:  # a balance bias works against popularity
            bias = (torch.randn(e, generator=gen, device="cuda") - popular) * (0.05 if case["score"] == "sigmoid" else 0.1 / e)
        for _ in range(50):
            rows = _unsure(case, logits, bias).nonzero()[:, 0]
            if rows.numel() == 0:
                break
            logits[rows] = (torch.randn(rows.numel(), e, generator=gen, device="cuda") * 1.5 + popular).to(logits.dtype)
        return {"case": case, "logits": logits, "bias": bias, "ids": new(t, k), "weights": new(t, k, dtype=torch.float32)}
    if op == "route_back":
        t, e, k = case["tokens"], case["experts"], case["k"]
        _, logits = _logits(case, gen)
        ids = logits.float().topk(k, 1).indices.to(torch.int32)
        grad = torch.randn(t, k, generator=gen, device="cuda")
        return {"case": case, "logits": logits, "ids": ids, "grad": grad, "grad_logits": torch.empty_like(logits)}
    if op == "group":
        n, e = case["slots"], case["groups"]
        skew = torch.rand(n, generator=gen, device="cuda")
        ids = (torch.where(skew < 0.5, skew * 2, torch.rand(n, generator=gen, device="cuda") ** 2) * e).long().clamp_(0, e - 1)
        ids = ids.to(torch.int32)
        if case["dropped"]:
            ids[torch.rand(n, generator=gen, device="cuda") < 0.03] = -1
        return {"case": case, "ids": ids, "offsets": new(e + 1), "order": new(n), "place": new(n)}
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if op == "weights":
        b, hq, h, q, s = (case[x] for x in ("batch", "q_heads", "kv_heads", "queries", "length"))
        w = torch.randn(b, hq, q, s, generator=gen, device="cuda").mul_(2.0).exp_()
        w.mul_(torch.arange(s, device="cuda") < lengths[:, None, None, None])
        w = w.div_(w.sum(3, keepdim=True)).to(TYPES[case["dtype"]])
        score = torch.rand(b, h, s, generator=gen, device="cuda") ** 4
        return {"case": case, "w": w, "score": score, "lengths": lengths, "out": torch.empty_like(score)}
    b, h, s, d, n = (case[x] for x in ("batch", "heads", "length", "width", "budget"))
    dtype = TYPES[case["dtype"]]
    # accumulated weights: a few entries hold most of it, some none at all
    score = torch.randn(b, h, s, generator=gen, device="cuda").mul_(2.0).sub_(6.0).exp_()
    score[torch.rand(b, h, s, generator=gen, device="cuda") < 0.05] = 0.0
    keys = torch.randn(b, h, s, d, generator=gen, device="cuda", dtype=dtype)
    values = torch.randn(b, h, s, d, generator=gen, device="cuda", dtype=dtype)
    return {"case": case, "score": score, "keys": keys, "values": values, "lengths": lengths,
            "keep": new(b, h, n), "kept": new(b), "out": (new(b, h, n, d, dtype=dtype), new(b, h, n, d, dtype=dtype),
                                                          new(b, h, n, dtype=torch.float32))}


# ------------------------------------------------------------ plain forms --

def _plain_scores(case, logits):
    x = logits.float()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_route(state):
    case, bias, k = state["case"], state["bias"], state["case"]["k"]
    s = _plain_scores(case, state["logits"])
    c = s if bias is None else s + bias
    if case["groups"] > 1:
        by = c.view(c.shape[0], case["groups"], -1)
        total = by.sort(dim=2, descending=True).values[:, :, :case["best"]].sum(2)
        at = total.sort(dim=1, descending=True, stable=True).indices[:, :case["picks"]]
        keep = torch.zeros_like(total, dtype=torch.bool).scatter_(1, at, True)
        c = torch.where(keep[:, :, None], by, -math.inf).flatten(1)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]


def _plain_route_back(state):
    case, ids, g = state["case"], state["ids"].long(), state["grad"] * state["case"]["scale"]
    s = _plain_scores(case, state["logits"])
    w = s.gather(1, ids)
    if case["renorm"]:  # through w / sum(w)
        total = w.sum(1, keepdim=True)
        g = (g - (g * w).sum(1, keepdim=True) / total) / total
    d = torch.zeros_like(s).scatter_(1, ids, g)
    if case["score"] == "softmax":
        d = s * (d - (g * w).sum(1, keepdim=True))
    else:
        d = d * s * (1.0 - s)
    return d.to(state["logits"].dtype)


def _plain_group(state):
    ids, e = state["ids"], state["case"]["groups"]
    key = torch.where((ids >= 0) & (ids < e), ids, e)
    key, order = key.sort(stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(key, torch.arange(e + 1, dtype=key.dtype, device=key.device)).to(torch.int32)
    return offsets, order.to(torch.int32), place.to(torch.int32)


def _plain_weights(state):
    case, w, score = state["case"], state["w"], state["score"]
    b, h, s = score.shape
    total = w.float().view(b, h, -1, s).sum(2) + case["decay"] * score
    return torch.where(torch.arange(s, device=w.device) < state["lengths"][:, None, None], total, 0.0)


def _plain_evict(state):
    case, score, n = state["case"], state["score"], state["lengths"][:, None, None]
    s, budget = case["length"], case["budget"]
    at = torch.arange(s, device=score.device).expand_as(score)
    tier = (at < n).int() + ((at < n) & ((at < case["first"]) | (at >= n - case["last"]))).int()
    order = torch.where(score.isnan(), -math.inf, score).sort(dim=2, descending=True, stable=True).indices
    order = order.gather(2, tier.gather(2, order).sort(dim=2, descending=True, stable=True).indices)[:, :, :budget]
    order = torch.where(tier.gather(2, order) > 0, order, s)
    if order.shape[2] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[2]), value=s)
    order = order.sort(dim=2).values
    there = order < s
    keep = torch.where(there, order, 0)
    b, h = score.shape[:2]
    row, head = torch.arange(b, device=score.device)[:, None, None], torch.arange(h, device=score.device)[:, None]
    new = [torch.where(there[..., None], x[row, head, keep], 0.0) for x in (state["keys"], state["values"])]
    kept = state["lengths"].clamp(max=budget)
    return (torch.where(there, keep, -1).to(torch.int32), kept, *new, torch.where(there, score.gather(2, keep), 0.0))


PLAIN = {"route": _plain_route, "route_back": _plain_route_back, "group": _plain_group, "weights": _plain_weights,
         "evict": _plain_evict}


# -------------------------------------------------------- the library's calls --

def _own(state):
    import ordered_merge_gb300 as om

    case, op = state["case"], state["case"]["op"]
    if op == "route":
        return om.route_topk(state["logits"], case["k"], score=case["score"], bias=state["bias"], groups=case["groups"],
                             group_picks=case["picks"], group_best=case["best"], renorm=case["renorm"],
                             scale=case["scale"], ids=state["ids"], weights=state["weights"])
    if op == "route_back":
        return om.route_topk_backward(state["logits"], state["ids"], state["grad"], score=case["score"],
                                      renorm=case["renorm"], scale=case["scale"], grad_logits=state["grad_logits"])
    if op == "group":
        return om.group_by_id(state["ids"], case["groups"], offsets=state["offsets"], order=state["order"],
                              place=state["place"])
    if op == "weights":
        return om.accumulate_weights(state["w"], state["score"], lengths=state["lengths"], decay=case["decay"],
                                     out=state["out"])
    keep, kept = om.evict_select(state["score"], case["budget"], first=case["first"], last=case["last"],
                                 lengths=state["lengths"], keep=state["keep"], kept=state["kept"])
    return (keep, kept, *om.evict_gather(keep, (state["keys"], state["values"], state["score"]), out=state["out"]))


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits --

def _exact_route(case, state):
    import numpy as np

    x = state["logits"].double().cpu().numpy()
    if case["score"] == "softmax":
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = np.reciprocal(1 + np.exp(-x))
    c = s.copy() if state["bias"] is None else s + state["bias"].double().cpu().numpy()
    rows, g = np.arange(len(x))[:, None], case["groups"]
    if g > 1:
        by = np.sort(c.reshape(len(x), g, -1), 2)[:, :, -case["best"]:].sum(2)
        out = np.argsort(-by, 1, kind="stable")[:, case["picks"]:]
        c.reshape(len(x), g, -1)[rows, out] = -np.inf
    ids = np.empty((len(x), case["k"]), np.int64)
    for j in range(case["k"]):  # argmax takes the first of equals
        ids[:, j] = c.argmax(1)
        c[rows[:, 0], ids[:, j]] = -np.inf
    w = s[rows, ids]
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return ids, w * case["scale"]


def _exact_route_back(case, state):
    with torch.enable_grad():  # the definition, differentiated
        x = state["logits"].detach().double().requires_grad_()
        s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
        w = torch.gather(s, 1, state["ids"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (w * case["scale"] * state["grad"].double()).sum().backward()
    return x.grad


def _exact_weights(case, state):
    b, h, s = state["score"].shape
    out = torch.zeros(b, h, s, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        for j in range(h):
            share = case["q_heads"] // h
            rows = state["w"][i, j * share:(j + 1) * share, :, :n].reshape(-1, n).double()
            out[i, j, :n] = case["decay"] * state["score"][i, j, :n].double() + rows.sum(0)
    return out


def _exact_group(case, state):
    import numpy as np

    ids, e = state["ids"].cpu().numpy(), case["groups"]
    order = np.concatenate([np.flatnonzero(ids == g) for g in range(e)] + [np.flatnonzero((ids < 0) | (ids >= e))])
    offsets = np.searchsorted(np.sort(ids[(ids >= 0) & (ids < e)]), np.arange(e + 1))
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    return offsets, order, place


def _exact_evict(case, state):
    import numpy as np

    score, n, budget = state["score"].cpu().numpy(), _lengths(case), case["budget"]
    b, h = score.shape[:2]
    keep = np.full((b, h, budget), -1, np.int64)
    for i in range(b):
        most = min(n[i], budget)
        fixed = np.zeros(n[i], bool)
        if n[i] <= budget:
            fixed[:] = True
        else:
            fixed[:case["first"]] = True
            fixed[n[i] - case["last"]:] = True
        for j in range(h):
            ranked = np.lexsort((np.arange(n[i]), -score[i, j, :n[i]].astype(np.float64), ~fixed))
            keep[i, j, :most] = np.sort(ranked[:most])
    at = torch.from_numpy(keep).to(state["score"].device)
    there, at = at >= 0, at.clamp(min=0)

    def moved(x):
        rows = torch.stack([x[i, j].index_select(0, at[i, j]) for i in range(b) for j in range(h)]).view(b, h, budget, -1)
        return (rows * there[..., None]).view(b, h, budget, *x.shape[3:])

    return keep, np.minimum(n, budget), moved(state["keys"]), moved(state["values"]), moved(state["score"])


def exact(case, seed):
    state = prepare(case, seed)
    return {"route": _exact_route, "route_back": _exact_route_back, "group": _exact_group, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](case, state)
