"""Plain 64-bit references of the ordered selections (numpy, row by row)."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U32 = 2.0 ** -24  # half an ulp of float32, relative


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def scores(x: np.ndarray, score: str) -> np.ndarray:
    """s of rows of logits; an expert at -inf or NaN has none."""
    x = np.where(np.isnan(x), -np.inf, x)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        top = x.max(1, keepdims=True)
        e = np.where(x == -np.inf, 0.0, np.exp(x - top))
        return e / e.sum(1, keepdims=True)


def choices(x, score, bias, by_logit=False):
    """What the experts of each row are ranked by; -inf where masked.  The logits themselves where their order
    decides (no bias, no sums over a group)."""
    s = x if by_logit else scores(x, score)
    c = s if bias is None else s + bias[None, :]
    open_ = (x > -np.inf) & (np.ones_like(x, bool) if bias is None else (bias > -np.inf)[None, :])
    return np.where(open_ & ~np.isnan(c), c, -np.inf)


def route(x, k, score="softmax", bias=None, groups=1, group_picks=1, group_best=1, renorm=False, scale=1.0):
    s, c = scores(x, score), choices(x, score, bias, bias is None and (groups == 1 or group_best == 1))
    n, e = x.shape
    ids, w = np.full((n, k), -1, np.int64), np.zeros((n, k))
    size = e // groups
    for t in range(n):
        if groups > 1:
            total = []
            for g in range(groups):
                best = sorted((v for v in c[t, g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:group_best]
                total.append((-sum(best), g) if best else (np.inf, g))
            live = [g for v, g in sorted(total)[:group_picks] if v < np.inf]
            for g in range(groups):
                if g not in live:
                    c[t, g * size:(g + 1) * size] = -np.inf
        ranked = sorted((-c[t, i], i) for i in range(e) if c[t, i] > -np.inf)[:k]
        for j, (_, i) in enumerate(ranked):
            ids[t, j] = i
        m = len(ranked)
        if m:
            if renorm:  # of the picked logits, shifted so that nothing underflows
                px = x[t, ids[t, :m]]
                with np.errstate(all="ignore"):
                    if score == "softmax":
                        p = np.exp(px - px.max())
                    else:
                        low = min(px.max(), 0.0)
                        p = np.exp(np.where(px >= 0, -np.log1p(np.exp(-np.abs(px))),
                                            px - np.log1p(np.exp(-np.abs(px)))) - low)
                w[t, :m] = p / p.sum()
            else:
                w[t, :m] = s[t, ids[t, :m]]
    return ids, w * scale


def route_backward(x, ids, grad, score="softmax", renorm=False, scale=1.0):
    """The gradient by the chain rule, slot by slot (Jacobian times vector)."""
    s = scores(x, score)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        live = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < x.shape[1] and x[t, ids[t, j]] > -np.inf]
        if not live:
            continue
        picked, g = ids[t, live], grad[t, live] * scale
        if renorm:
            _, w = route(x[t:t + 1, picked], len(live), score, renorm=True)
            back, _ = route(x[t:t + 1, picked], len(live), score, renorm=False)
            by_slot = np.empty(len(live))
            by_slot[back[0]] = w[0]
            jac = np.diag(by_slot) - np.outer(by_slot, by_slot)  # of softmax-like quotients, by log s
            d = jac @ g
            if score == "sigmoid":
                d = d * (1 - s[t, picked])
            out[t, picked] = d
        elif score == "sigmoid":
            out[t, picked] = g * s[t, picked] * (1 - s[t, picked])
        else:
            jac = np.diag(s[t]) - np.outer(s[t], s[t])
            full = np.zeros(x.shape[1])
            full[picked] = g
            out[t] = jac @ full
    return out


def group(ids, groups):
    ids = ids.reshape(-1)
    key = np.where((ids >= 0) & (ids < groups), ids.astype(np.int64), groups)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    return np.searchsorted(key[order], np.arange(groups + 1)), order, place


def evict(score, lengths, budget, first, last):
    b, h, s = score.shape
    keep = np.full((b, h, budget), -1, np.int64)
    for i in range(b):
        n = min(max(int(lengths[i]), 0), s)
        for j in range(h):
            row = np.where(np.isnan(score[i, j, :n]), -np.inf, score[i, j, :n])
            if n <= budget:
                chosen = np.arange(n)
            else:
                middle = np.arange(first, n - last)
                ranked = middle[np.argsort(-row[middle], kind="stable")][:budget - first - last]
                chosen = np.sort(np.concatenate([np.arange(first), ranked, np.arange(n - last, n)]))
            keep[i, j, :len(chosen)] = chosen
    return keep, np.minimum(np.clip(lengths, 0, s), budget)
