"""The sampled tree's acceptance in 64 bits, one node at a time, from its definition in
include/dfl2.h; host memory only."""
import numpy as np


def weights(cand, q, V):
    """A node's drafting weights by token; a repeated or impossible candidate counts as none."""
    d = {}
    for c, w in zip(cand, q):
        if 0 <= c < V and c not in d:
            d[int(c)] = float(w) if w > 0 else 0.0
    return d


def accept(p, tokens, parents, cand, q, u, replace):
    """One tree: p(i) -> the target's row at node i.  Returns path, next token."""
    T = len(tokens)
    path, V = [0], None
    while True:
        cur = path[-1]
        row = np.asarray(p(cur), np.float64)
        V = len(row)
        d = weights(cand[cur], q[cur], V)
        r = {x: row[x] for x in d}
        whole = max(0.0, 1.0 - sum(r.values()))
        rest, factor, took = whole, 1.0, None
        for c in range(cur + 1, T):
            x = int(tokens[c])
            if parents[c] != cur or d.get(x, 0.0) == 0.0:
                continue
            R, D = rest + sum(r.values()), sum(d.values())
            if float(u[c]) * d[x] * R < r[x] * D:
                took = c
                break
            r = {y: max(0.0, r[y] / R - d[y] / D) for y in r}
            rest, factor = rest / R, factor / R
            if not replace:
                d[x] = 0.0
            if rest + sum(r.values()) == 0.0:
                r, rest, factor = {y: row[y] for y in r}, whole, 1.0
                break
        if took is None:
            break
        path.append(took)
    left = row * factor
    for y in r:
        left[y] = r[y]
    if not left.sum() > 0:
        left = row
    run = np.cumsum(left)
    if not run[-1] > 0:
        return path, -1
    over = np.flatnonzero(run > float(u[0]) * run[-1])
    return path, int(over[0]) if len(over) else int(np.flatnonzero(left > 0)[-1])
