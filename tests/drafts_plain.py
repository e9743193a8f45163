"""Plain 64-bit implementations of the operators on drafted trees and chosen pages (numpy), written from
their definitions in include/mk.h, one row, node and head at a time."""
import math

import numpy as np


def lineage(parents):
    """Of each node: itself and its ancestors, nearest first, or None for an absent one."""
    got = []
    for i, p in enumerate(parents):
        if p == -1:
            got.append([i])
        elif 0 <= p < i and got[p] is not None:
            got.append([i] + got[p])
        else:
            got.append(None)
    return got


def tree_seen(n, parents, window=0):
    """[nodes, n + nodes] which slots each node sees, or None for an absent one."""
    rows = []
    for line in lineage(parents):
        if line is None:
            rows.append(None)
            continue
        depth = len(line) - 1
        seen = np.zeros(n + len(parents), dtype=bool)
        position = np.arange(n)
        seen[:n] = position > n + depth - window if window else True
        for up, j in enumerate(line):
            seen[n + j] = not window or up < window
        rows.append(seen)
    return rows


def accept(tokens, parents, choices):
    """The accepted nodes in order."""
    if parents[0] != -1:
        return []
    path = [0]
    while True:
        for i in range(path[-1] + 1, len(tokens)):
            if parents[i] == path[-1] and tokens[i] == choices[path[-1]]:
                path.append(i)
                break
        else:
            return path


def page_score(q, low, high):
    """The greatest product of a query head (of [heads, d]) with keys within the bounds [d]."""
    return max(math.fsum(max(x * a, x * b) for x, a, b in zip(h, low, high)) for h in q)


def choose(scores, pages, n_blocks, first, last):
    """The pages taken of `pages` many, in rising order."""
    if pages <= n_blocks:
        return list(range(pages))
    rank = [math.inf if math.isnan(s) else s for s in scores[:pages]]
    forced = [j for j in range(pages) if j < first or j >= pages - last]
    others = sorted((j for j in range(pages) if j not in forced), key=lambda j: (-rank[j], j))
    return sorted(forced + others[: n_blocks - len(forced)])
