"""Drawing a token from a row of logits, from the definition in float64."""

import numpy as np

FLOOR = 2.0 ** -40


def kept(x, temperature, top_k, top_p, min_p):
    """Indices that can be drawn, in index order, their weights, and how far
    the top-p cut is from taking one token more or less (relative)."""
    x = np.asarray(x, dtype=np.float64)
    order = np.lexsort((np.arange(len(x)), -x))      # value, then lower index
    with np.errstate(all="ignore"):
        w = np.exp((x[order] - x[order[0]]) / temperature)
    n = len(x)
    if 0 < top_k < n:
        n = top_k
    slack = 1.0
    if top_p < 1.0:
        goal = top_p * w[:n].sum()
        before = np.concatenate(([0.0], np.cumsum(w[:n])[:-1]))
        slack = float(np.abs(before[1:] - goal).min(initial=w[0])) / w[:n].sum()
        n = max(1, int((before < goal).sum()))
    n = max(1, int((w[:n] >= max(min(min_p, 1.0), FLOOR)).sum()))
    at = np.argsort(order[:n])
    return order[:n][at], w[:n][at], slack


def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability among the kept, distance from the nearest border
    between two tokens or two top-p cuts, relative to the total)."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x.max()) or np.isnan(x).any():
        return -1, np.nan, 1.0
    if temperature < 2.0 ** -100:
        return int(np.argmax(x)), 0.0, 1.0
    ids, w, slack = kept(x, temperature, top_k, top_p, min_p)
    run = np.cumsum(w)
    k = min(int(np.searchsorted(run, u * run[-1], side="right")), len(ids) - 1)
    borders = np.abs(np.concatenate(([0.0], run)) / run[-1] - u)
    borders[0] = 1.0 if u == 0 else borders[0]       # u = 0 is on the first token's side
    return int(ids[k]), float(np.log(w[k] / run[-1])), min(slack,
                                                           float(borders[:-1].min(initial=1.0)))


def walk(parent, tokens, target):
    """(path, emitted tokens) along the lowest-index matching children."""
    path = [0]
    while True:
        cur = path[-1]
        nxt = [i for i in range(1, len(parent))
               if (int(parent[i]) if 0 <= parent[i] < i else 0) == cur
               and target[cur] >= 0 and tokens[i] == target[cur]]
        if not nxt:
            break
        path.append(min(nxt))
    return path, [int(target[i]) for i in path]
