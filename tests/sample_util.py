"""The next token by temperature, top-k, top-p and min-p in float64 (numpy), with
how near the choice came to another one."""
import math

import numpy as np


def sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """-> (token, logprob, margin): margin is the smallest distance, relative to
    the sums, of any decision that a rounding could turn (the place of u in the
    running sum, the place of top_p, a weight's of min_p)."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    best = x.max()
    if best == -np.inf:
        return -1, -np.inf, 1.0
    if not t > 0:
        return int(x.argmax()), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == best, 1.0, 0.0) if best == np.inf else np.where(x > -np.inf, np.exp(np.where(x > -np.inf, x - best, 0) / t), 0.0)
    rank = np.lexsort((np.arange(x.size), -x))
    rank = rank[x[rank] > -np.inf]
    margin = 1.0
    if k > 0:
        rank = rank[:k]
    if p < 1:
        c = np.cumsum(w[rank])
        target = max(p, 0.0) * c[-1]
        n = min(int(np.searchsorted(c, target, side="left")), rank.size - 1) + 1
        if p > 0:
            margin = np.abs(c - target).min() / c[-1]
        rank = rank[:n]
    if m > 0:
        m = min(m, 1.0)
        if m < 1:
            margin = min(margin, np.abs(w[rank] - m).min())
        rank = rank[w[rank] >= m]
    kept = np.sort(rank)
    c = np.cumsum(w[kept])
    target = (u if u > 0 else 0.0) * c[-1]
    i = min(int(np.searchsorted(c, target, side="right")), kept.size - 1)
    while w[kept[i]] == 0:  # u of 1 and above: the last one that weighs something
        i -= 1
    if 0 < u < 1:
        margin = min(margin, np.abs(c - target).min() / c[-1])
    return int(kept[i]), math.log(w[kept[i]] / c[-1]), margin


def logits(rng, rows, vocab, kind, dtype):
    if kind == "flat":
        x = np.zeros((rows, vocab))
    elif kind == "steps":  # many ties
        x = rng.integers(-6, 7, (rows, vocab)) / 2.0
    elif kind == "one":
        x = rng.standard_normal((rows, vocab)) - 60
        x[np.arange(rows), rng.integers(0, vocab, rows)] = 5
    else:
        x = 2.2 * rng.standard_normal((rows, vocab))
        x[:, rng.integers(0, vocab, 1 + vocab // 3000)] += 6
        if kind == "masked":
            x[rng.random((rows, vocab)) < 0.9] = -np.inf
        if kind == "wide":
            x *= 1000
    return x.astype(dtype)
