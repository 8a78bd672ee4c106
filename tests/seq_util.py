"""Helpers of the causal-sequence tests: seeded inputs, and element by element how far
a kernel's output may be from the fp64 oracle.

Bounds, derived from the arithmetic the header states (u = eps/2 of the input type: half a
step of a rounding; products and sums in 32 bits):
  score error      es  = scale * D * 2^-22 * max_ij sum_d |q_id k_jd|   (fp32 sum of D products)
  lse              es + 2^-19 (1 + |lse|)                               (exp2 / log2 approximations)
  P, relative      rp  = 2 es + 2^-18 (1 + |lse|)
  out              (u [P as operand] + u [result] + rp) sum_j P|v|  (+ fp16: P below 2^-14
                   is held in steps of 2^-24, half of one per key: n 2^-25 max|v|)
  dS (before its rounding)  |dS| rp + P (es_dP + u sum_d |dO O| [delta uses the rounded O])
  gradients        the sums of (error + u |.|) of P or dS over the other operand, + u |result|
fp16 operands below 2^-14 again add half a step, 2^-25, per term.  Every bound gets 1 % for
the second-order terms left out.
"""
import numpy as np
import torch

from oracle import seq_oracle as O

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def f64(t):
    return t.detach().cpu().double().numpy()


def normal(rng, *shape, dtype, sigma=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(dtype)


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def score_error(q, k, scale):
    """Over all heads: the fp32 error bound of a score."""
    big = max([float(np.max(np.abs(q[:, h]) @ np.abs(k[:, h // (q.shape[1] // k.shape[1])]).T))
               for h in range(q.shape[1])] + [0.0]) if q.size and k.size else 0.0
    return scale * q.shape[2] * 2.0 ** -22 * big


def assert_close(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same_inf = np.isinf(want) & (got == want)
    off = np.where(same_inf, 0.0, np.abs(got - np.where(same_inf, 0.0, want)))
    off = np.where(same_inf, 0.0, off)
    bad = ~(off <= 1.01 * bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(off / (bound + 1e-300), nan=np.inf), 0.0)), off.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; at {i}: got {got[i]}, expected {want[i]}, "
                             f"bound {np.broadcast_to(bound, off.shape)[i]}")


def check_forward(q, k, v, out, lse, scale, dtype, what=""):
    """q [n,Hq,D], k, v [L,Hkv,D] fp64 of one sequence against the kernel's out [n,Hq,D], lse [Hq,n].
    Returns (oracle o, lse, w, p) and (rp [Hq, n])."""
    o, z, w, p = O.attend(q, k, v, scale)
    es, u = score_error(q, k, scale), U[dtype]
    fin = np.isfinite(z)
    zz = np.where(fin, np.abs(z), 0.0)
    assert_close(lse, z, es + 2.0 ** -19 * (1 + zz), f"{what} lse")
    rp = 2 * es + 2.0 ** -18 * (1 + zz)
    G = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        a = p[h] @ np.abs(v[:, h // G])
        vmax = np.max(np.abs(v[:, h // G]), initial=0.0)
        bound = (2 * u + rp[h][:, None]) * a + k.shape[0] * TINY[dtype] * vmax + TINY[dtype]
        assert_close(out[:, h], o[:, h], bound, f"{what} out head {h}")
    return (o, z, w, p), rp


def weight_bound(p, rp, group):
    """[Hkv, L] bound of the weights' error from p [Hq, n, L] and rp [Hq, n]."""
    per = np.einsum("hnl,hn->hl", p, rp + 2.0 ** -20 * p.shape[1] * group)
    return per.reshape(-1, group, p.shape[2]).sum(1) + 1e-30


def check_gradients(q, k, v, do, got, scale, dtype, what=""):
    """(dq, dk, dv) of one prompt against the oracle, element by element."""
    u, tiny = U[dtype], TINY[dtype]
    dq, dk, dv = O.gradients(q, k, v, do, scale)
    G, L, D = q.shape[1] // k.shape[1], k.shape[0], q.shape[2]
    bq, bk, bv = np.abs(dq) * u, np.abs(dk) * u, np.abs(dv) * u
    es = score_error(q, k, scale)
    for h in range(q.shape[1]):
        e = h // G
        o, z, p = O.rows_forward(q[:, h], k[:, e], v[:, e], 0, scale)
        rp = (2 * es + 2.0 ** -18 * (1 + np.where(np.isfinite(z), np.abs(z), 0.0)))[:, None]
        seen = np.tril(np.ones((L, L)))
        dp = do[:, h] @ v[:, e].T
        ds = np.abs(p * (dp - np.sum(do[:, h] * o, 1)[:, None]))
        edp = D * 2.0 ** -22 * (np.abs(do[:, h]) @ np.abs(v[:, e]).T)
        edelta = (u + D * 2.0 ** -22) * np.sum(np.abs(do[:, h] * o), 1)[:, None] + tiny * np.sum(np.abs(do[:, h]), 1)[:, None]
        # the rounded O also carries the forward's own rounding of P
        edelta += (u + rp) * (np.abs(do[:, h]) @ np.abs(v[:, e]).T * p).sum(1, keepdims=True)
        err = ds * (rp + u) + p * (edp + edelta) + tiny * seen
        bq[:, h] += scale * err @ np.abs(k[:, e])
        bk[:, e] += scale * err.T @ np.abs(q[:, h])
        bv[:, e] += (p * (rp + u) + tiny * seen).T @ np.abs(do[:, h])
    for name, g, w, b in (("dq", got[0], dq, bq), ("dk", got[1], dk, bk), ("dv", got[2], dv, bv)):
        assert_close(g, w, b + 2 * tiny + L * 2.0 ** -24 * np.max(np.abs(w), initial=0.0), f"{what} {name}")


def make_cache(rng, tables_for, page, kv_heads, D, dtype, spare=3, fill=float("nan")):
    """Pages for sequences of up to tables_for[b] places: (k_pages, v_pages, block_table); every
    element not written yet holds `fill`."""
    cols = max(1, max(-(-n // page) for n in tables_for))
    pages = len(tables_for) * cols + spare
    order = rng.permutation(pages)[:len(tables_for) * cols].astype(np.int32).reshape(len(tables_for), cols)
    k = torch.full((pages, page, kv_heads, D), fill, dtype=dtype)
    return k, k.clone(), torch.from_numpy(np.ascontiguousarray(order))


def fill_cache(k_pages, v_pages, table, b, k, v):
    """Rows k, v [L, Hkv, D] as places 0.. of sequence b (host tensors)."""
    page = k_pages.shape[1]
    j = torch.arange(k.shape[0])
    at = table[b].long()[j // page]
    k_pages[at, j % page] = k
    v_pages[at, j % page] = v
