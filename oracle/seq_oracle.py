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


def rotate(x, positions, inv_freq, interleaved=False, factor=1.0, inverse=False):
    """x [T, H, D], positions [T], inv_freq [R/2]: every feature pair as a complex number, times
    factor·exp(±i angle); features from R on unchanged."""
    R = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    turn = (factor * np.exp((-1j if inverse else 1j) * a))[:, None, :]
    out = np.array(x, np.float64)
    one, two = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = (out[..., one] + 1j * out[..., two]) * turn
    out[..., one], out[..., two] = z.real, z.imag
    return out


# What the codes 0 .. 126 of e4m3 stand for (127 is NaN; 128 + c is -c).
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def round_e4m3(x):
    """The nearest value of e4m3, of two the one of the even code; NaN stays NaN.  |x| <= 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), E4M3[-1])
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(x), np.nan, np.sign(x) * E4M3[code])


def scale8(most):
    """The least power of two s, 2^-64 at the least, with most <= 448 s."""
    s = 2.0 ** -64
    while most > 448.0 * s:
        s *= 2.0
    return s


def append8(codes, scales, new, first, block):
    """One sequence and head of keys or values of a cache in 8 bits, in place: codes [places, D] as the
    values they stand for, scales [places / block], new [n, D] from place first on."""
    end = first + len(new)
    for at in range(first // block * block, end, block):
        lo, hi = max(at, first), min(at + block, end)
        rows = np.where(np.isfinite(new[lo - first:hi - first]), new[lo - first:hi - first], np.nan)
        s = scale8(np.nanmax(np.abs(rows), initial=0.0) if np.isfinite(rows).any() else 0.0)
        if lo > at:
            s = max(s, scales[at // block])
            codes[at:lo] = round_e4m3(codes[at:lo] * (scales[at // block] / s))
        codes[lo:hi] = round_e4m3(rows / s)
        scales[at // block] = s
