"""GPU: attention over the 8-bit cache where weights and scales lie far apart, and over long contexts with flat scores, against the
fp64 oracle within bounds that follow from the weights themselves (tests/seq8_util.py, close_bounds; what they notice:
tests/test_seq8_checks.py).  Every way of the attention: few rows a key; many in place
(one tile of queries, two), as a table too wide for a copy makes them; many over a copy."""
import numpy as np
import pytest
import torch

from memory_efficient_biased_gb300 import evo_attn as E
from memory_efficient_biased_gb300 import evo_seq as Q
from oracle import seq_oracle as O
from tests import seq8_util as C
from tests import seq_util as S

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
WAYS = ["few", "one tile", "two tiles", "copied"]


def attend(way, cache, ctx, q, Hk, scale=None):
    """(out, lse) of the new tokens q [n, Hq, D] of one sequence, and that the call goes that way."""
    n, Hq, D = q.shape
    rows, cols = n * Hq // Hk, cache.table.shape[1]
    assert rows <= 32 if way == "few" else rows > 512 if way == "copied" else 32 < rows <= 512
    table = cache.table
    if way in ("one tile", "two tiles"):  # 2^28 values, and more, of each of keys and values
        table = torch.full((1, (1 << 28) // (Hk * D * cache.page) + 1), -1, dtype=torch.int32, device="cuda")
        table[:, :cols] = cache.table
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [ctx]))
    args = q.cuda(), *cache.args(), cu, lens, table
    out, lse = Q.evo_paged8_fwd(*args, scale=scale)
    again = Q.evo_paged8_fwd(*args, scale=scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert E.evo_attn_device_status() == 0
    return S.f64(out), S.f64(lse)


def tokens_of(way, G):
    return {"few": 32 // G, "one tile": 32 // G + 1, "two tiles": 512 // G, "copied": 512 // G + 1}[way]


@pytest.mark.parametrize("apart", [12, 20, 40, 88])
@pytest.mark.parametrize("order", ["large first", "small first", "mixed"])
@pytest.mark.parametrize("way", WAYS)
def test_blocks_of_equal_weight_and_scales_far_apart(way, order, apart):
    """All keys alike (the same weight); half of the blocks have a scale 2^apart times the others' and codes of 0 in half of
    the features: there the small blocks' values are all that there is.  (Few rows: an item that is not cut, several blocks a warp.)"""
    rng = np.random.default_rng(apart)
    Hq, Hk, D, ctx = 8, 2, 64, 1000 if way == "few" else 1500
    n = -(-ctx // 16)
    large = rng.random(n) < 0.5 if order == "mixed" else (np.arange(n) < n // 2) == (order == "large first")

    def v(b, length):
        x = O.round_e4m3(rng.uniform(1.0, 440.0, (length, Hk, D)))
        x[np.repeat(large, 16)[:length], :, :D // 2] = 0.0
        return x, np.repeat(np.where(large, 2.0 ** (apart // 2), 2.0 ** (apart // 2 - apart))[:, None], Hk, 1)

    cache = C.coded(rng, [ctx], 64, 16, Hk, D, lambda b, length: (np.zeros((length, Hk, D)), np.ones((n, Hk))), v)
    q = S.normal(rng, tokens_of(way, Hq // Hk), Hq, D, dtype=BF)
    out, lse = attend(way, cache, ctx, q, Hk)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, D ** -0.5, BF, way == "few", way)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("way", ["few", "one tile", "copied"])
def test_one_key_of_large_weight_and_scale(way, dtype):
    """One key with 2^13 times the weight and 2^12 times the scale of each of the others, and codes of 0 in half of the features."""
    rng = np.random.default_rng(3)
    Hq, Hk, D, ctx = 8, 1, 64, 20000 if way == "copied" else 131071
    big, sign, n = ctx // 2 + 5, np.where(rng.random(D) < 0.5, -1.0, 1.0), -(-ctx // 16)

    def k(b, length):
        x = np.zeros((length, Hk, D))
        x[big] = 9.0 * sign
        return x, np.ones((n, Hk))

    def v(b, length):
        x, s = O.round_e4m3(rng.uniform(1.0, 4.0, (length, Hk, D))), np.full((n, Hk), 2.0 ** -4)
        at = big // 16 * 16
        s[at // 16] = 2.0 ** 8
        x[at:at + 16] = 0.0
        x[big, :, D // 2:] = 3.0
        return x, s

    cache = C.coded(rng, [ctx], 128, 16, Hk, D, k, v)
    q = torch.from_numpy(np.ascontiguousarray(np.broadcast_to(sign / (9.0 * D), (tokens_of(way, Hq), Hq, D)), np.float32)).to(dtype)
    scale = float(np.float32(13 * np.log(2.0)))
    out, lse = attend(way, cache, ctx, q, Hk, scale)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, scale, dtype, way == "few", way)


@pytest.mark.parametrize("dtype,lo,hi", [(BF, -44, 45), (FP, -14, 8), (FP, -33, 8), (FP, -33, -23)])
@pytest.mark.parametrize("D,page,block", [(64, 64, 16), (128, 16, 16), (96, 128, 64)])
@pytest.mark.parametrize("way", WAYS)
def test_scales_of_any_size(way, D, page, block, dtype, lo, hi):
    """Every block of values has a scale of its own, anywhere in the range; half of the codes are 0; scores spread over 30 powers
    of two."""
    rng = np.random.default_rng(D + page)
    Hq, Hk, ctx = 8, 2, 1000 if way == "few" else 1777
    n = -(-ctx // block)
    make = lambda zeros, s: lambda b, length: (  # noqa: E731
        O.round_e4m3(rng.standard_normal((length, Hk, D)) * 20.0) * (rng.random((length, Hk, D)) >= zeros), s)
    cache = C.coded(rng, [ctx], page, block, Hk, D, make(0.0, 2.0 ** rng.integers(-6, -3, (n, Hk))),
                    make(0.5, 2.0 ** rng.integers(lo, hi, (n, Hk))))
    q = S.normal(rng, tokens_of(way, Hq // Hk), Hq, D, dtype=dtype, sigma=3.0)
    out, lse = attend(way, cache, ctx, q, Hk)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, D ** -0.5, dtype, way == "few", way)


@pytest.mark.parametrize("way", WAYS)
def test_queries_with_one_large_feature(way):
    """bf16 queries with a feature 2^20 times the others, where the keys have nothing: the others make the scores."""
    rng = np.random.default_rng(6)
    Hq, Hk, D, ctx = 8, 2, 128, 700
    n = -(-ctx // 32)

    def k(b, length):
        x = O.round_e4m3(rng.standard_normal((length, Hk, D)))
        x[:, :, 17] = 0.0
        return x, np.ones((n, Hk))

    cache = C.coded(rng, [ctx], 32, 32, Hk, D, k, lambda b, length: (O.round_e4m3(rng.standard_normal((length, Hk, D))), np.ones((n, Hk))))
    q = S.normal(rng, tokens_of(way, Hq // Hk), Hq, D, dtype=BF)
    q[:, :, 17] = 2.0 ** 20
    out, lse = attend(way, cache, ctx, q, Hk)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, D ** -0.5, BF, way == "few", way)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("way,ctx", [("few", 131071), ("few", 70003), ("one tile", 131071), ("two tiles", 30011), ("copied", 30011)])
def test_long_flat_contexts(way, ctx, dtype):
    """Contexts over every SM, every tile with a part in the result that cannot be missed."""
    rng = np.random.default_rng(ctx)
    Hq, Hk, D = 8, 1, 64
    k, v = C.flat_rows(rng, ctx, D)
    ones = np.ones((-(-ctx // 64), Hk))
    cache = C.coded(rng, [ctx], 64, 64, Hk, D, lambda b, n: (k[:, None], ones * 2.0 ** -5), lambda b, n: (v[:, None], ones))
    q = S.normal(rng, tokens_of(way, Hq), Hq, D, dtype=dtype)
    out, lse = attend(way, cache, ctx, q, Hk)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, D ** -0.5, dtype, way == "few", way)


def test_long_flat_contexts_together():
    """Several of them of uneven lengths in a call, items and pieces on every SM."""
    rng = np.random.default_rng(12)
    Hq, Hk, D, ctx = 4, 2, 64, [9001, 40007, 128, 17, 22222]
    flat = [[C.flat_rows(rng, n, D) for _ in range(Hk)] for n in ctx]
    ones = lambda n, s: np.full((-(-n // 16), Hk), s)  # noqa: E731
    cache = C.coded(rng, ctx, 16, 16, Hk, D, lambda b, n: (np.stack([x[0] for x in flat[b]], 1), ones(n, 2.0 ** -5)),
                    lambda b, n: (np.stack([x[1] for x in flat[b]], 1), ones(n, 1.0)))
    for chunks in ([1] * 5, [9, 30, 5, 17, 60]):
        q = S.normal(rng, sum(chunks), Hq, D, dtype=BF)
        lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), lens, cache.table)
        a = 0
        for b, n in enumerate(chunks):
            C.check_close(S.f64(q[a:a + n]), *cache.rows(b, ctx[b]), S.f64(out[a:a + n]), S.f64(lse[:, a:a + n]), D ** -0.5, BF,
                          chunks[0] == 1, f"sequence {b}")
            a += n
    assert E.evo_attn_device_status() == 0


@pytest.mark.parametrize("power", [-60, -20, 40, 100])
@pytest.mark.parametrize("way", WAYS)
def test_scales_far_from_one(way, power):
    """All scales of values alike and far from 1: the log-sum-exp, and P, know nothing of them.  Contexts of a few keys (a wide range of
    lse's relative precision), and ones that are cut."""
    rng = np.random.default_rng(100 + power)
    Hq, Hk, D = 8, 2, 64
    for ctx in (1, 7, 900, 5000):
        n = -(-ctx // 16)
        cache = C.coded(rng, [ctx], 64, 16, Hk, D, lambda b, length: (O.round_e4m3(rng.standard_normal((length, Hk, D))), np.full((n, Hk), 2.0 ** -6)),
                        lambda b, length: (O.round_e4m3(rng.standard_normal((length, Hk, D)) * 9), np.full((n, Hk), 2.0 ** power)))
        tokens = tokens_of(way, Hq // Hk)
        q = S.normal(rng, tokens, Hq, D, dtype=BF)
        out, lse = attend(way, cache, ctx, q, Hk)
        see = min(ctx, tokens)  # (more tokens than keys: the first of them see none)
        C.check_close(S.f64(q)[tokens - see:], *cache.rows(0, ctx), out[tokens - see:], lse[:, tokens - see:], D ** -0.5, BF, way == "few", way)
        assert np.all(out[:tokens - see] == 0) and np.all(lse[:, :tokens - see] == -np.inf)


def test_fp16_many_keys_of_small_weight_and_scale():
    """In front of each head's keys one of 2^17.5 times the weight and 2^20 times the scale of each of the others, whose values are all
    that there is in half of the features.  (More heads than SMs: one reference for most of a head's keys.)"""
    rng = np.random.default_rng(8)
    Hk, G, D, ctx = 160, 8, 64, 4096
    sign, n = np.where(rng.random(D) < 0.5, -1.0, 1.0), ctx // 16

    def k(b, length):
        x = np.zeros((length, Hk, D))
        x[3] = 9.0 * sign
        return x, np.ones((n, Hk))

    def v(b, length):
        x, s = np.repeat(O.round_e4m3(rng.uniform(200.0, 440.0, (length, 1, D))), Hk, 1), np.full((n, Hk), 2.0 ** -20)
        s[0] = 1.0
        x[:16] = 0.0
        x[3, :, D // 2:] = 3.0
        return x, s

    cache = C.coded(rng, [ctx], 128, 16, Hk, D, k, v)
    q = torch.from_numpy(np.ascontiguousarray(np.broadcast_to(sign / (9.0 * D), (tokens_of("one tile", G), G * Hk, D)), np.float32)).to(FP)
    scale = float(np.float32(17.5 * np.log(2.0)))
    out, lse = attend("one tile", cache, ctx, q, Hk, scale)
    C.check_close(S.f64(q), *cache.rows(0, ctx), out, lse, scale, FP, False)
