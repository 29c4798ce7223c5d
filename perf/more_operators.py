"""Cases for measuring the operators of a decoding step and of the embedding.

Five operators, beside the ordered selections that they work with:

  beam        the best continuations of a beam search, from the logits and the
              beams' cumulative log probabilities
  reorder     the beams' caches moved to the beams that go on
  embed       rows of an embedding table by token, scaled; and its gradient,
              the rows of equal tokens summed
  experts     a layer of routed experts for the few tokens of a decoding step

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

def _beam(name, batch, beams, vocab, top, dtype, masked=0.0, finished=0.0):
    return {"name": name, "op": "beam", "batch": batch, "beams": beams, "vocab": vocab, "top": top, "dtype": dtype,
            "masked": masked, "finished": finished}


def _reorder(name, batch, beams, heads, capacity, width, prompt, dtype):
    return {"name": name, "op": "reorder", "batch": batch, "beams": beams, "heads": heads, "capacity": capacity,
            "width": width, "prompt": prompt, "dtype": dtype}


def _embed(name, tokens, rows, width, dtype, scale):
    return {"name": name, "op": "embed", "tokens": tokens, "rows": rows, "width": width, "dtype": dtype, "scale": scale}


def _embed_back(name, tokens, rows, width, dtype, into, scale):
    return {"name": name, "op": "embed_back", "tokens": tokens, "rows": rows, "width": width, "dtype": dtype,
            "into": into, "scale": scale}


def _experts(name, tokens, experts, top, hidden, inner, gated, act, dtype):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "top": top, "hidden": hidden,
            "inner": inner, "gated": gated, "act": act, "dtype": dtype}


def listed():
    return [
        # one prompt, four beams, twice as many continuations as beams: the smallest call, all latency
        _beam("beam-one-prompt", 1, 4, 32768, 8, "bf16"),
        # a batch in 32 bits with forbidden tokens and a few beams that have ended; a vocabulary of odd size
        _beam("beam-batch", 16, 5, 50021, 10, "f32", 0.02, 0.1),
        # a server's batch over a large vocabulary of odd size
        _beam("beam-server", 64, 8, 131071, 16, "bf16"),
        # one prompt's caches of one layer, a few hundred tokens in
        _reorder("reorder-one-prompt", 1, 4, 8, 1024, 128, 500, "bf16"),
        # a batch of long prompts: what all beams of a prompt share stays where it is
        _reorder("reorder-batch", 8, 8, 8, 4096, 128, 1000, "bf16"),
        # the tokens of 64 decoding sequences
        _embed("embed-decode", 64, 131072, 4096, "bf16", 64.0),
        # a long prefill
        _embed("embed-prefill", 65536, 131072, 2048, "bf16", 1.0),
        # the gradient of a microbatch
        _embed_back("embed-back-microbatch", 4096, 32768, 1024, "bf16", "bf16", 32.0),
        # the gradient of a large batch of odd length into 32 bits, for an optimizer that keeps them
        _embed_back("embed-back-batch", 65537, 131072, 2048, "bf16", "f32", 1.0),
        # one token through 8 of 64 gated experts
        _experts("experts-one-token", 1, 64, 8, 2048, 1024, True, "silu", "bf16"),
        # a few tokens through plain experts whose sizes are no powers of two
        _experts("experts-few", 12, 32, 4, 2000, 1400, False, "gelu", "f16"),
        # 64 decoding sequences through 8 of 128 gated experts: nearly all of them are read
        _experts("experts-batch", 64, 128, 8, 2048, 1024, True, "silu", "bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["beam", "beam", "reorder", "embed", "embed_back", "embed_back", "experts", "experts"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "beam":
        beams, vocab = rng.randint(1, 16), _spread(rng, 500, 131072)
        batch = _spread(rng, 1, max(1, min(64, 64 * 8 * 131071 * 2 // (beams * vocab * SIZE[dtype]))))
        case = _beam("", batch, beams, vocab, rng.randint(1, 2 * beams), dtype, rng.choice([0.0, 0.02, 0.995]),
                     rng.choice([0.0, 0.2]))
    elif op == "reorder":
        beams, heads, width = rng.randint(2, 16), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128])
        capacity = _spread(rng, 16, 4096)
        most = 8 * 8 * 8 * 4096 * 128 * 2 // (beams * heads * width * capacity * SIZE[dtype])
        case = _reorder("", _spread(rng, 1, max(1, min(8, most))), beams, heads, capacity, width,
                        rng.randint(0, capacity // 2), dtype)
    elif op == "embed":
        width = rng.choice([_spread(rng, 32, 4096), 64 * rng.randint(1, 64)])
        tokens = _spread(rng, 1, min(65536, 65536 * 2048 * 2 // (width * SIZE[dtype])))
        case = _embed("", tokens, _spread(rng, 200, 131072), width, dtype, rng.choice([1.0, width ** 0.5]))
    elif op == "embed_back":
        width = rng.choice([_spread(rng, 32, 4096), 64 * rng.randint(1, 64)])
        into = rng.choice([dtype, "f32"])
        tokens = _spread(rng, 1, min(65536, 65536 * 2048 * 2 // (width * SIZE[dtype])))
        rows = _spread(rng, 200, min(131072, 131072 * 2048 * 4 // (width * SIZE[into])))
        case = _embed_back("", tokens, rows, width, dtype, into, rng.choice([1.0, width ** 0.5]))
    else:
        hidden, inner = 8 * _spread(rng, 16, 512), 8 * _spread(rng, 8, 256)
        gated, size = rng.random() < 0.6, 2
        experts = _spread(rng, 4, max(4, min(256, 128 * 1024 * 2048 * 3 // (hidden * inner * 3))))
        top = rng.randint(1, min(8, experts))
        case = _experts("", _spread(rng, 1, 64), experts, top, hidden, inner, gated, rng.choice(["silu", "gelu", "relu"]),
                        rng.choice(["bf16", "f16"]))
    case.pop("name")
    return case


def _alive(case):
    """Beams of a sequence that go on: some twice or more, the others of them not."""
    return max(1, (case["beams"] * 5 + 7) // 8)


def _lengths(case):
    """Entries of each sequence's cache; the first is full.  Those of the prompt are the same for all its beams."""
    return [case["capacity"] - (b * 2654435761) % (case["capacity"] // 4 + 1) for b in range(case["batch"])]


def _distinct(n, kinds, power):
    """How many of `kinds` are expected among n draws of floor(kinds * u ** power)."""
    import numpy as np

    edge = (np.arange(kinds + 1) / kinds) ** (1 / power)
    return float(-np.expm1(n * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12))).sum())


def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "beam":  # the logits of the beams that have not ended, the scores; scores, parents and tokens out
        rows = case["batch"] * case["beams"]
        read = rows - _ended(case) * case["batch"]
        return {"bytes": read * case["vocab"] * size + rows * 5 + case["batch"] * case["top"] * 12,
                "flops": 5 * read * case["vocab"]}
    if op == "reorder":  # keys and values of the beams that go on in, of all beams out
        entries = sum(n - min(n, case["prompt"]) for n in _lengths(case)) * case["heads"]
        return {"bytes": 2 * entries * case["width"] * size * (_alive(case) + case["beams"])
                + case["batch"] * (case["beams"] + 2) * 4, "flops": 0}
    if op == "embed":
        n, w = case["tokens"], case["width"]
        return {"bytes": (n + _distinct(n, case["rows"], POWER)) * w * size + n * 8, "flops": n * w}
    if op == "embed_back":
        n, w = case["tokens"], case["width"]
        return {"bytes": n * w * size + case["rows"] * w * SIZE[case["into"]] + n * 8, "flops": n * w}
    t, k, h, i = case["tokens"], case["top"], case["hidden"], case["inner"]
    mats = 3 if case["gated"] else 2
    touched = case["experts"] * (1 - (1 - k / case["experts"]) ** t)  # expected
    return {"bytes": touched * mats * h * i * size + 2 * t * h * size + t * k * 8, "flops": 2 * t * k * h * i * mats}


# ----------------------------------------------------------------- inputs --

POWER = 4.0  # tokens are floor(rows * u ** POWER): the first are frequent, as in a vocabulary ordered by frequency


def _ended(case):
    return int(case["beams"] * case["finished"] + 0.5)


def _continuations(case, state):
    """Every continuation's score in 64 bits, [batch, beams * vocab]."""
    x = state["logits"].double()
    x = torch.where(x.isnan(), -math.inf, x)
    lse = torch.logsumexp(x, 2, keepdim=True)
    c = torch.where(x > -math.inf, state["scores"].double()[:, :, None] + (x - lse), -math.inf)
    c[state["finished"]] = -math.inf
    c[:, :, case["end"]] = torch.where(state["finished"], state["scores"].double(), c[:, :, case["end"]])
    return c.flatten(1)


def _unsure(case, state):
    """Sequences whose choice hangs on the rounding of a logarithm: continuations of two beams closer than a
    few parts in a million.  Either order is right there, so their scores are drawn anew."""
    v, at = _continuations(case, state).topk(min(case["top"] + 1, case["beams"] * case["vocab"]), 1)
    other = at[:, 1:] // case["vocab"] != at[:, :-1] // case["vocab"]
    near = (v[:, :-1] - v[:, 1:]).abs() < 1e-5 * (1 + v[:, :-1].abs())
    return (other & near & torch.isfinite(v[:, 1:])).any(1)


def _tokens(case, gen):
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    return (u ** POWER * case["rows"]).long().clamp_(max=case["rows"] - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    randn = lambda *shape, **kw: torch.randn(*shape, generator=gen, device="cuda", **kw)  # noqa: E731
    new = lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "beam":
        b, n, v, k = (case[x] for x in ("batch", "beams", "vocab", "top"))
        case = dict(case, end=2)
        logits = randn(b, n, v, dtype=dtype).mul_(2.5)
        logits += (randn(b, 1, v) * 1.5).to(dtype)  # beams of a sequence agree on much
        if case["masked"]:
            logits.masked_fill_(torch.rand(b, n, v, generator=gen, device="cuda") < case["masked"], -math.inf)
        finished = torch.rand(b, n, generator=gen, device="cuda").argsort(1) < _ended(case)
        state = {"case": case, "logits": logits, "finished": finished, "out": (new(b, k, dtype=torch.float32), new(b, k), new(b, k))}
        draw_scores = lambda m: (randn(m, n).abs_().mul_(1.5) + 12.0).neg_().sort(1, descending=True).values  # noqa: E731
        state["scores"] = draw_scores(b)
        for _ in range(20):
            rows = _unsure(case, state).nonzero()[:, 0]
            if rows.numel() == 0:
                break
            state["scores"][rows] = draw_scores(rows.numel())
        return state
    if op == "reorder":
        b, n, h, s, d = (case[x] for x in ("batch", "beams", "heads", "capacity", "width"))
        # the beams that go on, each at least once, in the order of their continuations' scores
        live = torch.rand(b, n, generator=gen, device="cuda").argsort(1)[:, :_alive(case)]
        more = live.gather(1, torch.randint(0, _alive(case), (b, n - _alive(case)), generator=gen, device="cuda"))
        parents = torch.cat([live, more], 1)
        parents = parents.gather(1, torch.rand(b, n, generator=gen, device="cuda").argsort(1)).to(torch.int32)
        lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        caches = [randn(b, n, h, s, d, dtype=dtype) for _ in range(2)]
        return {"case": case, "parents": parents.contiguous(), "caches": caches, "lengths": lengths,
                "starts": lengths.clamp(max=case["prompt"]), "out": [torch.zeros_like(x) for x in caches]}
    if op == "embed":
        ids = _tokens(case, gen)
        table = randn(case["rows"], case["width"], dtype=dtype)
        return {"case": case, "ids": ids, "table": table, "out": new(case["tokens"], case["width"], dtype=dtype)}
    if op == "embed_back":
        ids = _tokens(case, gen)
        if case["tokens"] > 8:
            ids[-(case["tokens"] // 8):] = -1  # the padding at the end of a batch
        return {"case": case, "ids": ids, "grad": randn(case["tokens"], case["width"], dtype=dtype),
                "grad_table": new(case["rows"], case["width"], dtype=TYPES[case["into"]])}
    t, e, k, h, i = (case[x] for x in ("tokens", "experts", "top", "hidden", "inner"))
    mats = lambda rows, cols: randn(e, rows, cols, dtype=dtype).mul_(cols ** -0.5)  # noqa: E731
    ids = torch.rand(t, e, generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32)
    weights = torch.softmax(randn(t, k), 1)
    return {"case": case, "x": randn(t, h, dtype=dtype), "ids": ids.contiguous(), "weights": weights, "up": mats(i, h),
            "gate": mats(i, h) if case["gated"] else None, "down": mats(h, i), "out": new(t, h, dtype=dtype)}


# ------------------------------------------------------------ plain forms --

def _plain_beam(state):
    case, ended = state["case"], state["finished"]
    vocab, end, k = case["vocab"], case["end"], case["top"]
    x = state["logits"].float()
    m = x.amax(2, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    lse = m + torch.log(torch.exp(x - m).sum(2, keepdim=True))
    # the sum in 64 bits: two logits next to each other would often tie in 32
    scores = state["scores"].double()
    c = torch.where(x > -math.inf, scores[:, :, None] + (x.double() - lse.double()), -math.inf)
    c = torch.where(ended[:, :, None], -math.inf, c)
    c[:, :, end] = torch.where(ended, scores, c[:, :, end])
    best, at = c.flatten(1).sort(dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    there = best > -math.inf
    return (best.float(), torch.where(there, at // vocab, -1).to(torch.int32),
            torch.where(there, at % vocab, -1).to(torch.int32))


def _plain_reorder(state):
    case, parents = state["case"], state["parents"].long()
    row = torch.arange(case["batch"], device=parents.device)[:, None]
    at = torch.arange(case["capacity"], device=parents.device)
    moved = (at >= state["starts"][:, None]) & (at < state["lengths"][:, None])
    return [torch.where(moved[:, None, None, :, None], x[row, parents], o) for x, o in zip(state["caches"], state["out"])]


def _plain_embed(state):
    return (state["table"][state["ids"]].float() * state["case"]["scale"]).to(state["table"].dtype)


def _plain_embed_back(state):
    case, ids = state["case"], state["ids"]
    there = (ids >= 0) & (ids < case["rows"])
    total = torch.zeros(case["rows"] + 1, case["width"], device=ids.device)
    total.index_add_(0, torch.where(there, ids, case["rows"]), state["grad"].float())
    return (total[:-1] * case["scale"]).to(TYPES[case["into"]])


def _plain_act(act, x):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))
    return x * (x > 0)


def _plain_experts(state):
    case, x, k = state["case"], state["x"].float(), state["case"]["top"]
    e = state["ids"].long().flatten()
    rows = x.repeat_interleave(k, 0)[:, :, None]
    a = (state["up"][e].float() @ rows)[:, :, 0]
    if case["gated"]:
        a = _plain_act(case["act"], (state["gate"][e].float() @ rows)[:, :, 0]) * a
    else:
        a = _plain_act(case["act"], a)
    y = (state["down"][e].float() @ a[:, :, None])[:, :, 0]
    y = (y.view(len(x), k, -1) * state["weights"][:, :, None]).sum(1)
    return y.to(state["x"].dtype)


PLAIN = {"beam": _plain_beam, "reorder": _plain_reorder, "embed": _plain_embed, "embed_back": _plain_embed_back,
         "experts": _plain_experts}


# -------------------------------------------------------- the library's calls --

def _own(state):
    import ordered_merge_gb300 as om

    case, op = state["case"], state["case"]["op"]
    if op == "beam":
        scores, parents, tokens = state["out"]
        return om.beam_select(state["logits"], case["top"], state["scores"], finished=state["finished"],
                              end_id=case["end"], out_scores=scores, parents=parents, tokens=tokens)
    if op == "reorder":
        return om.beam_gather(state["parents"], state["caches"], starts=state["starts"], lengths=state["lengths"],
                              out=state["out"])
    if op == "embed":
        return om.embed_lookup(state["ids"], state["table"], scale=case["scale"], out=state["out"])
    if op == "embed_back":
        return om.embed_lookup_backward(state["grad"], state["ids"], case["rows"], scale=case["scale"],
                                        grad_table=state["grad_table"])
    return om.expert_mlp(state["x"], state["ids"], state["weights"], state["up"], state["down"], gate=state["gate"],
                         act=case["act"], out=state["out"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits --

def _exact_beam(case, state):
    case, k = state["case"], case["top"]
    out = []
    for b in range(case["batch"]):
        one = {x: state[x][b:b + 1] for x in ("logits", "scores", "finished")}
        c = _continuations(case, one)[0]
        edge = c.topk(min(k, c.numel())).values[-1]
        at = ((c >= edge) & (c > -math.inf)).nonzero()[:, 0]
        at = at[c[at].sort(descending=True, stable=True).indices[:k]]
        room = k - at.numel()
        out.append((torch.nn.functional.pad(c[at], (0, room), value=-math.inf),
                    torch.nn.functional.pad(at // case["vocab"], (0, room), value=-1),
                    torch.nn.functional.pad(at % case["vocab"], (0, room), value=-1)))
    return tuple(torch.stack(x) for x in zip(*out))


def _exact_reorder(case, state):
    out = [x.clone() for x in state["out"]]
    for b, n in enumerate(_lengths(case)):
        lo = min(n, case["prompt"])
        for j, p in enumerate(state["parents"][b].tolist()):
            for x, o in zip(state["caches"], out):
                o[b, j, :, lo:n] = x[b, p, :, lo:n]
    return out


def _exact_embed(case, state):
    return torch.index_select(state["table"], 0, state["ids"]).double() * case["scale"]


def _exact_embed_back(case, state):
    out = torch.zeros(case["rows"], case["width"], dtype=torch.float64, device="cuda")
    there = state["ids"] >= 0
    ids, order = state["ids"][there].sort()
    grad = state["grad"][there][order].double()
    for lo in range(0, len(ids), 8192):
        out.index_add_(0, ids[lo:lo + 8192], grad[lo:lo + 8192], alpha=case["scale"])
    return out


def _exact_experts(case, state):
    x, y = state["x"].double(), torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}[case["act"]]
    for e in range(case["experts"]):
        t, j = (state["ids"] == e).nonzero(as_tuple=True)
        if t.numel():
            a = torch.nn.functional.linear(x[t], state["up"][e].double())
            if case["gated"]:
                a = act(torch.nn.functional.linear(x[t], state["gate"][e].double())) * a
            else:
                a = act(a)
            y[t] += torch.nn.functional.linear(a, state["down"][e].double()) * state["weights"][t, j].double()[:, None]
    return y


def exact(case, seed):
    state = prepare(case, seed)
    return {"beam": _exact_beam, "reorder": _exact_reorder, "embed": _exact_embed, "embed_back": _exact_embed_back,
            "experts": _exact_experts}[case["op"]](case, state)
