"""Eviction in plain Python, from its definition: on a CacheModel and a float array of weights."""
import math

import numpy as np


def order_key(w):
    """Descending weight, NaN first, -0 as 0; equal ones by place."""
    return (0, 0.0) if math.isnan(w) else (1, -(w + 0.0))


def evict(model, weights, slots, keep, recent, sinks):
    """weights [layers, slots, heads, places]; returns the status bits, and changes nothing unless
    they are 0."""
    if not model._valid(slots) or len(set(slots)) < len(slots):
        return 1
    for s, n in zip(slots, keep):
        if n < recent + sinks:
            return 2
        if model.lengths[s] > n:
            for i in range(sinks // model.ps, model.pages_of(n)):
                if model.refs[model.table[s][i]] != 1:
                    return 8
    layers, _, heads, _, _ = model.k.shape
    for s, n in zip(slots, keep):
        length = model.lengths[s]
        if length <= n:
            continue
        gap, last = n - recent, length - recent
        for layer in range(layers):
            for h in range(heads):
                w = weights[layer, s, h]
                ranked = sorted(range(sinks, last), key=lambda j: order_key(float(w[j])))
                stays = set(ranked[:gap - sinks])
                holes = [j for j in range(sinks, gap) if j not in stays]
                above = [j for j in range(gap, last) if j in stays]
                to = holes + list(range(gap, n))
                frm = above + list(range(last, length))
                a = [model.place(s, t) for t in to]
                b = [model.place(s, t) for t in frm]
                for x in (model.k, model.v):
                    rows = [x[layer, p, h, r].copy() for p, r in b]
                    for (p, r), row in zip(a, rows):
                        x[layer, p, h, r] = row
                w[to] = w[frm].copy() if frm else w[to]
                w[n:length] = 0
        model._drop(s, n)
    return 0


def random_weights(rng, shape, kind):
    """Spread ones, ones with many ties, and ones with zeros, negatives, infinities and NaN."""
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    w = rng.gamma(0.3, 2.0, shape).astype(np.float32)
    if kind == "odd":
        for value in (0.0, -0.0, -1.5, np.inf, -np.inf, np.nan, 1e-40, -1e-40):
            w[rng.random(shape) < 0.06] = value
    return w
