"""Routing of tokens to experts in numpy, in 64 bits, one token at a time."""
import numpy as np


def scores(kind, l):
    l = l.astype(np.float64)
    with np.errstate(over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def route(kind, logits, topk, bias=None, groups=1, keep=1, group_top=1, renormalize=False,
          scale=1.0):
    """(picks, weights): -1 and 0 where fewer than topk experts can be picked."""
    tokens, experts = logits.shape
    picks = np.full((tokens, topk), -1, np.int32)
    weights = np.zeros((tokens, topk))
    size = experts // groups
    for t, l in enumerate(logits):
        s = scores(kind, l)
        c = s + (0 if bias is None else bias.astype(np.float64))
        if bias is None and groups == 1:
            c = l.astype(np.float64)  # the same order
        c = np.where(l == -np.inf, -np.inf, c)
        open_ = np.ones(experts, bool)
        if groups > 1:
            score = []
            for g in range(groups):
                best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_top]
                best = best[best > -np.inf]
                score.append(best.sum() if len(best) else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
            open_ = np.isin(np.arange(experts) // size, kept)
        can = [e for e in range(experts) if open_[e] and c[e] > -np.inf]
        order = sorted(can, key=lambda e: (-c[e], e))[:topk]
        picks[t, :len(order)] = order
        w = s[order]
        if renormalize and len(order):
            if kind == "softmax":
                e = np.exp(l[order].astype(np.float64) - l[order].max())
                w = e / e.sum()
            else:
                w = w / w.sum() if w.sum() > 0 else w * 0
        weights[t, :len(order)] = w * scale
    return picks, weights


def route_backward(kind, logits, picks, dweights, renormalize, scale):
    """(dlogits, the sum of the magnitudes of what is added up)."""
    out, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    for t, l in enumerate(logits):
        s = scores(kind, l)
        on = [(e, j) for j, e in enumerate(picks[t]) if 0 <= e < len(l) and l[e] > -np.inf]
        e = [x for x, _ in on]
        g = dweights[t, [j for _, j in on]].astype(np.float64) * scale
        if not e:
            continue
        if renormalize:
            if kind == "softmax":
                p = np.exp(l[e].astype(np.float64) - l[e].max())
            else:
                p = s[e]
            p = p / p.sum() if p.sum() > 0 else p * 0
            d, m = p * (g - (g * p).sum()), p * (np.abs(g) + (np.abs(g) * p).sum())
            rest = 1 / (1 + np.exp(l[e].astype(np.float64))) if kind == "sigmoid" else 1.0
            out[t, e], mag[t, e] = d * rest, m * rest
        elif kind == "sigmoid":
            out[t, e] = g * s[e] / (1 + np.exp(l[e].astype(np.float64)))
            mag[t, e] = np.abs(out[t, e])
        else:
            full = np.zeros(len(l))
            full[e] = g
            out[t] = s * (full - (g * s[e]).sum())
            mag[t] = s * (np.abs(full) + (np.abs(g) * s[e]).sum())
    return out, mag


def plan(picks, first, groups):
    """(offsets, sources, places): pairs sorted by expert, in their order inside each."""
    e = picks.reshape(-1).astype(np.int64) - first
    pairs = np.flatnonzero((e >= 0) & (e < groups))
    order = pairs[np.argsort(e[pairs], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(e[pairs], minlength=groups))])
    sources = np.full(e.size, -1, np.int32)
    sources[:order.size] = order
    places = np.full(e.size, -1, np.int32)
    places[order] = np.arange(order.size)
    return offsets[:groups + 1].astype(np.int64), sources, places
