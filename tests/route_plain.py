"""Plain 64-bit forms of routing, of the sort by expert and of the router's
gradient, token by token, and the bounds that the GPU results are held to."""
import math

import numpy as np

F32 = 2.0 ** -24          # half a step, relative to the value
F16 = 2.0 ** -11


def scores(x, score):
    """fp64 scores of one row of logits."""
    x = np.asarray(x, dtype=np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max()
    if top == -np.inf:
        return np.zeros_like(x)
    with np.errstate(invalid="ignore"):
        e = np.exp(x - top)
        return e / e.sum()


def choose(x, k, bias, score, groups=1, top_groups=1, group_best=1):
    """ids of one row: the rule as it is documented, one expert after another."""
    x = np.asarray(x, dtype=np.float64)
    E = len(x)
    by_score = bias is not None or (groups > 1 and group_best == 2)
    key = scores(x, score) if by_score else x.copy()
    if bias is not None:
        key = key + np.asarray(bias, dtype=np.float64)
    key = [math.inf if math.isnan(v) else v for v in key]
    key = [-math.inf if x[e] == -math.inf else key[e] for e in range(E)]
    if groups > 1:
        size, rank = E // groups, []
        for g in range(groups):
            part = sorted(key[g * size:(g + 1) * size], reverse=True)[:group_best]
            live = [v for v in part if v > -math.inf]
            rank.append(sum(live) if live else -math.inf)
        keep = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
        key = [key[e] if e // size in keep else -math.inf for e in range(E)]
    order = sorted(range(E), key=lambda e: (-key[e], e))[:k]
    return [e if key[e] > -math.inf else -1 for e in order] + [-1] * max(0, k - E)


def weights(x, ids, score, renorm, scale):
    s = scores(x, score)
    w = np.array([s[e] if e >= 0 else 0.0 for e in ids])
    if renorm:
        # the same quotient, where all of the scores underflow
        xs = np.array([x[e] for e in ids if e >= 0], dtype=np.float64)
        if len(xs):
            top = xs.max()
            v = np.exp(xs - top) if score == "softmax" else \
                np.exp(np.minimum(xs, 0) - min(top, 0)) / (1 + np.exp(-np.abs(xs)))
            w[[e >= 0 for e in ids]] = v / v.sum()
    return scale * w


def weight_bound(x, ref):
    """Half a step for each of: the shift by the largest logit (relative to the
    exponent), the exponential (two steps), at most 22 additions of the sum, the
    quotient and the scale; twice, for the quotient's two sides.  A result below
    fp32's normal range may be off by its smallest normal number."""
    x = np.asarray(x, dtype=np.float64)
    live = x[np.isfinite(x)]
    spread = min(104.0, live.max() - live.min()) if len(live) else 0.0
    return np.abs(ref) * F32 * 2 * (2 * spread + 32) + 2.0 ** -126 * (1 + len(x))


def rows(ids, E):
    """offsets and place of ids (T, k)."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    nxt, place = offsets[:-1].astype(np.int64).copy(), np.full(flat.shape, -1, dtype=np.int32)
    for i, e in enumerate(flat):
        if 0 <= e < E:
            place[i] = nxt[e]
            nxt[e] += 1
    return offsets, place.reshape(np.shape(ids))


def grad(x, ids, dw, score, renorm, scale):
    """dx of one row, by the formulas."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, score)
    live = [j for j, e in enumerate(ids) if 0 <= e < len(x) and x[e] != -np.inf]
    dx = np.zeros_like(x)
    if not live:
        return dx
    e = np.array([ids[j] for j in live])
    g = scale * np.asarray(dw, dtype=np.float64)[live]
    if renorm:
        r = weights(x, list(e), score, True, 1.0)
        d = r * (g - (r * g).sum())
        if score == "sigmoid":
            d *= 1.0 / (1.0 + np.exp(x[e]))
        np.add.at(dx, e, d)
    elif score == "sigmoid":
        np.add.at(dx, e, g * s[e] / (1.0 + np.exp(x[e])))
    else:
        full = np.zeros_like(x)
        np.add.at(full, e, g)
        dx = s * (full - (full * s).sum())
    return dx


def grad_bound(x, ids, dw, ref, score, renorm, scale, half_step):
    """The weights' bound times what each gradient is made of, and the last rounding.

    dx_e is a difference of terms of the size of g and of sum |g_j| w_j, each with
    the weights' relative error (and 2 k more half steps for the sums over the
    choices), times a weight of that error again."""
    x = np.asarray(x, dtype=np.float64)
    live = x[np.isfinite(x)]
    spread = min(104.0, live.max() - live.min()) if len(live) else 0.0
    rel = F32 * (4 * (2 * spread + 32) + 4 * len(ids) + 44)
    ok = [j for j, e in enumerate(ids) if 0 <= e < len(x) and x[e] != -np.inf]
    g = np.abs(scale * np.asarray(dw, dtype=np.float64))
    size = np.zeros_like(x)
    if ok:
        e = np.array([ids[j] for j in ok])
        full = np.zeros_like(x)
        np.add.at(full, e, g[ok])
        if renorm:
            w = np.zeros_like(x)
            np.add.at(w, e, weights(x, list(e), score, True, 1.0))
            size = w * (full + (full * w).sum())
        else:
            s = scores(x, score)
            size = s * full if score == "sigmoid" else s * (full + (full * s).sum())
    return rel * size + half_step * np.abs(ref) + (2.0 ** -25 if half_step == F16 else 0.0) + 2.0 ** -120
