"""Plain fp64 CPU oracle of the causal-sequence operators (include/evo_seq.h):
attention over packed prompts and its gradients, attention of new tokens over
a paged cache with the sums of its weights, and eviction by those sums.

TEST INFRASTRUCTURE ONLY, like ``evo_oracle``; it shares no code with the CUDA
library.  Sequences are numpy arrays here: offsets, pages and tables are resolved by
the caller.

Pins: tests/test_seq_oracle.py (differences, a loop over single scores, closed
forms and invariants).
"""
from __future__ import annotations

import numpy as np


def rows_forward(q, k, v, first, scale):
    """One head: n rows q [n, D] at positions first + i over keys k, v [L, D], row i seeing
    the keys j <= first + i.  Returns (o [n, D], lse [n], p [n, L])."""
    n, L = q.shape[0], k.shape[0]
    o, lse, p = np.zeros(q.shape), np.full(n, -np.inf), np.zeros((n, L))
    for i in range(n):
        seen = min(max(first + i + 1, 0), L)
        if seen == 0:
            continue
        x = scale * (k[:seen] @ q[i])
        m = np.max(x)
        e = np.exp(x - m)
        total = np.sum(e)
        p[i, :seen] = e / total
        lse[i] = m + np.log(total)
        o[i] = p[i, :seen] @ v[:seen]
    return o, lse, p


def attend(q, k, v, scale):
    """Grouped heads: q [n, Hq, D] the last n of the L tokens of k, v [L, Hkv, D].
    Returns (o [n, Hq, D], lse [Hq, n], w [Hkv, L]: P summed over rows and a group's heads,
    p [Hq, n, L])."""
    n, Hq, D = q.shape
    L, Hk = k.shape[0], k.shape[1]
    o, lse, w, ps = np.zeros(q.shape), np.zeros((Hq, n)), np.zeros((Hk, L)), np.zeros((Hq, n, L))
    for h in range(Hq):
        e = h // (Hq // Hk)
        o[:, h], lse[h], ps[h] = rows_forward(q[:, h], k[:, e], v[:, e], L - n, scale)
        w[e] += ps[h].sum(0)
    return o, lse, w, ps


def gradients(q, k, v, do, scale):
    """Gradients of <O, dO> of a whole prompt (n = L): (dq, dk, dv)."""
    Hq, Hk = q.shape[1], k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for h in range(Hq):
        e = h // (Hq // Hk)
        o, _, p = rows_forward(q[:, h], k[:, e], v[:, e], k.shape[0] - q.shape[0], scale)
        dp = do[:, h] @ v[:, e].T
        ds = p * (dp - np.sum(do[:, h] * o, axis=1)[:, None])
        dq[:, h] = scale * (ds @ k[:, e])
        dk[:, e] += scale * (ds.T @ q[:, h])
        dv[:, e] += p.T @ do[:, h]
    return dq, dk, dv


def choose(weights, length, budget, recent):
    """The places that stay of one sequence and head, in order."""
    if length <= budget:
        return list(range(length))
    old = range(length - recent)
    value = [(-np.inf, 1) if np.isnan(weights[j]) else (weights[j], 0) for j in old]
    # larger weights first, a NaN behind every number, the older of two equal ones first
    order = sorted(old, key=lambda j: (-value[j][0], value[j][1], j))
    return sorted(order[:budget - recent]) + list(range(length - recent, length))
