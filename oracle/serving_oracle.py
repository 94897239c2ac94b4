"""fp64 CPU oracle of what happens between two decode steps: drafts verified
against the target's probabilities, request lists rewritten, a pool made
contiguous.  Plain loops, written from the operators' words; test
infrastructure only."""
import math

import numpy as np


def _prob(x):
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=1.0, neginf=0.0)
    return np.clip(x, 0.0, 1.0)


def verify(target, tokens, uniforms, draft=None, parents=None):
    """target [B, W, V] -> path [B, W], accepted [B], next token [B], and whether a token or parent was bad."""
    B, W, V = target.shape
    path = np.full((B, W), -1, dtype=np.int64)
    accepted = np.zeros(B, dtype=np.int64)
    following = np.zeros(B, dtype=np.int64)
    bad = set()
    for b in range(B):
        up = [-1] + list(range(W - 1)) if parents is None else [int(x) for x in parents[b]]
        for i in range(W):
            if not -1 <= up[i] < i:
                bad.add("tree")
                up[i] = -1
            if i and not 0 <= tokens[b, i] < V:
                bad.add("token")
        walk = [0]
        while True:
            node, left, gone = walk[-1], 1.0, []
            row = _prob(target[b, node])
            for c in range(1, W):
                if up[c] != node:
                    continue
                x = int(tokens[b, c])
                inside = 0 <= x < V
                t = float(row[x]) if inside and x not in [int(tokens[b, g]) for g in gone] else 0.0
                against = left if draft is None else float(_prob(draft[b, c, x])) if inside else 0.0
                u = float(uniforms[b, c])
                if (u if u > 0 else 0.0) * against < t:
                    walk.append(c)
                    break
                left = max(left - t, 0.0)
                gone.append(c)
            else:
                break
        if gone and draft is not None:
            row = np.maximum(row - _prob(draft[b, gone[0]]), 0.0)
        for g in gone if draft is None else []:
            if 0 <= tokens[b, g] < V:
                row[int(tokens[b, g])] = 0.0
        run = np.cumsum(row)
        u, some = float(uniforms[b, 0]), np.nonzero(row > 0)[0]
        if not len(some):
            following[b] = -1
        else:
            past = np.nonzero(run > u * run[-1])[0] if not math.isnan(u) else []
            past = [v for v in past[:1]]
            following[b] = past[0] if past and row[past[0]] > 0 else (some[0] if past else some[-1])
        path[b, :len(walk)] = walk
        accepted[b] = len(walk)
    return path, accepted, following, bad


def repack(indptr, indices, sources, path=None, accepted=None):
    """New lists (one array of slots a request) and the slots that they give up, ascending."""
    rows = []
    for s in sources:
        if not 0 <= s < len(indptr) - 1:
            rows.append([])
            continue
        mine = [int(x) for x in indices[indptr[s]:indptr[s + 1]]]
        if path is not None and len(mine) >= path.shape[1]:
            w = path.shape[1]
            mine = mine[:len(mine) - w] + [mine[len(mine) - w + int(i)] for i in path[s][:accepted[s]]]
        rows.append(mine)
    old = {int(x) for x in indices[:indptr[-1]]}
    return rows, sorted(old - {x for mine in rows for x in mine})


def compact(indices):
    """Number of live slots, and where each of them goes that moves."""
    live = sorted({int(x) for x in indices})
    n, there = len(live), set(live)
    return n, dict(zip([x for x in live if x >= n], [x for x in range(n) if x not in there]))
