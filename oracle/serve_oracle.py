"""Float64 oracle of the routing and of the low-rank adapters, from the formulas in
include/exl3.h.  Plain numpy; test infrastructure."""
import numpy as np


def logits(x, weight, bias=None):
    """x weight^T (+ bias), and sum |x| |weight| (+ |bias|) for error bounds."""
    x, weight = np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    y, mag = x @ weight.T, np.abs(x) @ np.abs(weight).T
    if bias is not None:
        y, mag = y + bias.astype(np.float64), mag + np.abs(bias.astype(np.float64))
    return y, mag


def scores(l, scoring):
    """softmax or sigmoid of one token's logits."""
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        p = np.exp(l - (np.nan if np.isnan(l).any() else l.max()))
        return p / p.sum()


def _best(values, count):
    """Places of the `count` best values, best first: ties to the lower, NaN last."""
    return sorted(range(len(values)), key=lambda e: (bool(np.isnan(values[e])), -values[e], e))[:count]


def route(logits, topk, scoring="softmax", balance=None, groups=1, topk_groups=None, group_score="max",
          renormalize=True, scale=1.0):
    """ids [t, topk] and weights [t, topk]."""
    logits = np.asarray(logits, dtype=np.float64)
    t, e = logits.shape
    size, topk_groups = e // groups, groups if topk_groups is None else topk_groups
    ids, weights = np.zeros((t, topk), dtype=np.int64), np.zeros((t, topk))
    for i, l in enumerate(logits):
        s = scores(l, scoring)
        v = l if balance is None else s + np.asarray(balance, dtype=np.float64)
        members = list(range(e))
        if topk_groups < groups:
            grades = []
            for g in range(groups):
                mine = (s if group_score == "top2" and balance is None else v)[g * size:(g + 1) * size]
                top = mine[_best(mine, 2 if group_score == "top2" else 1)]
                with np.errstate(invalid="ignore"):
                    grades.append(top.sum())
            kept = sorted(_best(np.array(grades), topk_groups))
            members = [g * size + j for g in kept for j in range(size)]
        chosen = [members[j] for j in _best(v[members], topk)]
        w = s[chosen]
        with np.errstate(invalid="ignore", divide="ignore"):
            weights[i] = scale * (w / w.sum() if renormalize else w)
        ids[i] = chosen
    return ids, weights


def lora(x, a, b, rows, base=None, scales=None, ranks=None):
    """y, and what bounds its error (all without the scale's rounding): the adapter's
    sums of magnitudes sum_j |b_j| sum |a_j| |x|, and sum_j |b_j| times the largest of
    sum |a_j| |x| over j."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    m, n = x.shape[0], b.shape[1]
    y = np.zeros((m, n)) if base is None else np.array(base, dtype=np.float64)
    mag, peak = np.zeros((m, n)), np.zeros((m, n))
    with np.errstate(invalid="ignore", over="ignore"):
        for i, adapter in enumerate(rows):
            if not 0 <= adapter < a.shape[0]:
                continue
            r = a.shape[1] if ranks is None else int(np.clip(ranks[adapter], 0, a.shape[1]))
            s = 1.0 if scales is None else float(scales[adapter])
            y[i] += s * (b[adapter, :, :r] @ (a[adapter, :r] @ x[i]))
            sizes = np.abs(a[adapter, :r]) @ np.abs(x[i])
            mag[i] = abs(s) * (np.abs(b[adapter, :, :r]) @ sizes)
            peak[i] = abs(s) * np.abs(b[adapter, :, :r]).sum(-1) * (sizes.max() if r else 0.0)
    return y, mag, peak
