"""Beam search's selection and state moves on the host, from their definition:
every candidate's score in fp64, sorted; rows moved one by one."""

import numpy as np


def select(logits, scores, n, finished=None, end_id=0):
    """logits [G, K, V], scores [G, K] -> (scores fp64, parents, tokens) [G, n]."""
    x = np.asarray(logits, dtype=np.float64)
    c = np.asarray(scores, dtype=np.float64)
    G, K, V = x.shape
    out = np.full((G, K, V), -np.inf)
    with np.errstate(all="ignore"):
        for g in range(G):
            for k in range(K):
                if not abs(c[g, k]) <= 2e9:
                    continue
                if finished is not None and finished[g][k]:
                    out[g, k, end_id] = c[g, k]
                    continue
                row = x[g, k]
                lse = np.max(row) + np.log(np.sum(np.exp(row - np.max(row))))
                if np.isfinite(lse):
                    out[g, k] = c[g, k] + (row - lse)
    flat = out.reshape(G, K * V)
    at = np.argsort(-flat, axis=1, kind="stable")[:, :n]
    return np.take_along_axis(flat, at, 1), at // V, at % V


def reorder(pool, slot_ids, parents):
    """pool [P, S, C] -> (the pool after the move, the new slot ids)."""
    new_pool, new_ids = pool.copy(), np.array(slot_ids).copy()
    for g, (ids, par) in enumerate(zip(np.array(slot_ids), np.array(parents))):
        free = [int(ids[b]) for b in range(len(ids)) if b not in set(par.tolist())]
        seen = set()
        for j, p in enumerate(par.tolist()):
            slot = int(ids[p]) if p not in seen else free.pop(0)
            seen.add(p)
            new_ids[g, j] = slot
            new_pool[:, slot] = pool[:, ids[p]]
    return new_pool, new_ids
