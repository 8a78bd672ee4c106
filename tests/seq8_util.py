"""Helpers of the tests of the 8-bit cache: a cache on the host, what its codes stand for, and how
far attention over it may be from the fp64 oracle.

Appending and reading have no tolerance: every rounding is stated (nearest even, powers of two as
scales), so codes and scales are equal to the oracle's.

Attention, bounds as in tests/seq_util.py with k and v the values the codes stand for (they enter
the products exactly): es the error of a score in 32 bits, rp = 2 es + 2^-18 (1 + |lse|) the relative
one of P, and for the result
    (u_P [P as an operand in fp16 or dtype: at most half a step of dtype] + u [result] + rp) sum P|v|
    + keys 2^-25 2 max|v| [fp16's smallest step: P times its block's scale, taken against the largest such
      product, is held in steps of 2^-24; a code is at most 448, and 448 scale at most 2 max|v|
      where scales are the least that fit; given scales: 448 max scale].
"""
import numpy as np
import torch

from oracle import seq_oracle as O
from tests import seq_util as S

E4M3 = torch.float8_e4m3fn


def value_of(pages, scales):
    """What a cache's codes [P, page, H, D] stand for, in fp64, from scales [P, H, page / block]."""
    p, page, h, d = pages.shape
    n = scales.shape[2]
    v = pages.view(torch.uint8).cpu().numpy()
    c = v & 127
    x = np.where(c == 127, np.nan, O.E4M3[np.minimum(c, 126)]) * np.where(v & 128, -1.0, 1.0)
    s = scales.double().cpu().numpy().transpose(0, 2, 1)[:, :, None, :, None]
    return (x.reshape(p, n, page // n, h, d) * s).reshape(p, page, h, d)


class Cache:
    """A cache of sequences of up to places[b] tokens, on the GPU; codes not written are NaN, scales -7."""

    def __init__(self, rng, places, page, block, heads, D, spare=3, interleaved=False):
        cols = max(1, max(-(-n // page) for n in places))
        n = len(places) * cols + spare
        order = rng.permutation(n)[:len(places) * cols].astype(np.int32).reshape(len(places), cols)
        self.page, self.block, self.table = page, block, torch.from_numpy(np.ascontiguousarray(order)).cuda()
        if interleaved:
            both = torch.full((n, 2, page, heads, D), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = (torch.full((n, page, heads, D), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3) for _ in "kv")
        self.ks, self.vs = (torch.full((n, heads, page // block), -7.0, device="cuda") for _ in "kv")

    def args(self):
        return self.k, self.v, self.ks, self.vs

    def rows(self, b, length):
        """What places 0 .. length - 1 of sequence b hold: (k, v) [length, H, D] fp64."""
        j = np.arange(length)
        at = self.table[b].cpu().numpy()[j // self.page]
        return tuple(value_of(x, s)[at, j % self.page] for x, s in ((self.k, self.ks), (self.v, self.vs)))

    def fill(self, b, k, v, scale=None):
        """Rows k, v [L, H, D] fp64 as places 0 .. of sequence b, quantised on the host; scale(rows) gives
        a block's own scale [H], by default the least power of two that fits."""
        least = lambda x: np.array([O.scale8(np.max(np.abs(x[:, h]))) for h in range(x.shape[1])])  # noqa: E731
        table = self.table[b].cpu().numpy()
        for pages, scales, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
            for at in range(0, len(x), self.block):
                rows = x[at:at + self.block]
                s = (scale or least)(rows)
                p, i = int(table[at // self.page]), at % self.page
                codes = torch.from_numpy(O.round_e4m3(np.clip(rows / s[None, :, None], -448, 448))).to(E4M3)
                pages[p, i:i + len(rows)].view(torch.uint8).copy_(codes.view(torch.uint8))
                scales[p, :, i // self.block] = torch.from_numpy(s).float().cuda()


def check_attention(q, k, v, out, lse, scale, dtype, what="", vmax=None):
    """q [n,Hq,D], k, v [L,Hkv,D] fp64 of one sequence against out [n,Hq,D], lse [Hq,n]; vmax: see above."""
    o, z, _, p = O.attend(q, k, v, scale)
    es, u = S.score_error(q, k, scale), S.U[dtype]
    zz = np.where(np.isfinite(z), np.abs(z), 0.0)
    S.assert_close(lse, z, es + 2.0 ** -19 * (1 + zz), f"{what} lse")
    rp = 2 * es + 2.0 ** -18 * (1 + zz)
    G = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        big = 2 * np.max(np.abs(v[:, h // G]), initial=0.0) if vmax is None else vmax
        bound = (2 * u + rp[h][:, None]) * (p[h] @ np.abs(v[:, h // G])) + k.shape[0] * 2.0 ** -25 * big + S.TINY[dtype]
        S.assert_close(out[:, h], o[:, h], bound, f"{what} out head {h}")


def coded(rng, ctx, page, block, heads, D, k, v, **kw):
    """A Cache of sequences of ctx[b] tokens that holds what k(b, n) and v(b, n) give: (values [n, H, D] that are
    numbers of e4m3, scales [ceil(n / block), H]), written as they are."""
    cache = Cache(rng, ctx, page, block, heads, D, **kw)
    for b, n in enumerate(ctx):
        j = torch.arange(n, device="cuda")
        at = cache.table[b].long()[j // page]
        first = torch.arange(0, n, block, device="cuda")
        first_at = cache.table[b].long()[first // page]
        for pages, scales, make in ((cache.k, cache.ks, k), (cache.v, cache.vs, v)):
            x, s = make(b, n)
            codes = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(E4M3)
            pages.view(torch.uint8)[at, j % page] = codes.view(torch.uint8)
            scales[first_at, :, first % page // block] = torch.from_numpy(np.ascontiguousarray(s, np.float32)).cuda()
    return cache


def close_bounds(q, k, v, z, p, scale, dtype, few):
    """How far out [n,Hq,D] and lse [Hq,n] may be off, from the weights themselves: sharper than check_attention, whose
    last term takes the largest weight as 1 and every code as 448.  z, p: the oracle's lse and weights; few: the
    kernel for few rows a key.

    P is rounded by u_P: to fp16 (few), to dtype otherwise.  What is below fp16's normal numbers is held in steps of 2^-24:
      few   the largest P s_v of a row is held as 2^14.  Keys of 16 next to each other share their scale and
            are held against their own largest weight, as 2^13 to 2^14, where they lie 2^14 or more below the row's largest and their
            scale 2^4 or more below the largest so far; otherwise theirs is 1 or more: half a step is 2^-25 of the 16's largest
            weight at the most.  Where their scale is not that much smaller it is 2^-25 2^-14 2^4 of the row's largest weight
      many  fp16 alone: 2^-25 of the largest weight (the reference is at most the row's maximum)
    times |v| of each key.  With fp16 and many rows values are in steps of 2^-24 too.  bf16 queries lose what is below 2^-39 of their row's largest."""
    es, u = S.score_error(q, k, scale), S.U[dtype]
    G = q.shape[1] // k.shape[1]
    if dtype == torch.bfloat16:
        most = max(float(np.max(np.abs(k[:, h]).sum(-1))) for h in range(k.shape[1]))
        es += scale * 2.0 ** -39 * float(np.max(np.abs(q))) * most
    zz = np.where(np.isfinite(z), np.abs(z), 0.0)
    rp = 2 * es + 2.0 ** -18 * (1 + zz)
    out = np.zeros(q.shape)
    for h in range(q.shape[1]):
        a, w = np.abs(v[:, h // G]), p[h]
        bound = ((2.0 ** -11 if few else u) + u + rp[h][:, None]) * (w @ a) + S.TINY[dtype]
        if few:
            pad = -len(a) % 16
            blocks = np.pad(a, ((0, pad), (0, 0))).reshape(-1, 16, a.shape[1]).sum(1)
            most = np.pad(w, ((0, 0), (0, pad))).reshape(len(w), -1, 16).max(2)
            bound = bound + 2.0 ** -25 * (most @ blocks) + 2.0 ** -35 * w.max(1)[:, None] * a.sum(0)
        elif dtype == torch.float16:
            bound = bound + 2.0 ** -25 * w.max(1)[:, None] * a.sum(0) + 2.0 ** -25
        out[:, h] = bound
    return out, es + 2.0 ** -19 * (1 + zz)


def check_close(q, k, v, out, lse, scale, dtype, few, what=""):
    """check_attention with the bounds above."""
    o, z, _, p = O.attend(q, k, v, scale)
    bound, lse_bound = close_bounds(q, k, v, z, p, scale, dtype, few)
    S.assert_close(lse, z, lse_bound, f"{what} lse")
    S.assert_close(out, o, bound, f"{what} out")


def flat_rows(rng, n, D):
    """Keys [n, D] of e4m3 whose scores lie close together, and values that are positive in the features of their own
    tile of 128 keys and 0 in the others, so that each tile alone makes a good part of some features (D of 2 a tile):
    no tile can be left out, or counted twice, without that."""
    tile = np.arange(n) // 128
    v = np.where((np.arange(D)[None] % (D // 2)) == (tile % (D // 2))[:, None], rng.uniform(1.0, 2.0, (n, D)), 0.0)
    return O.round_e4m3(rng.standard_normal((n, D))), O.round_e4m3(v)
