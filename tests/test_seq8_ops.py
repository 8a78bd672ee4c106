"""GPU: rotary positions and the 8-bit cache against the fp64 oracle (bounds: tests/seq8_util.py, and
beside each test): odd sizes, parts of a head, far positions, blocks begun and gone on with, values
that are not finite, rows that see nothing, strided rows and pages, bad offsets, lengths and pages,
streams and captured graphs, and runs of them together with the attention."""
import numpy as np
import pytest
import torch

from memory_efficient_biased_gb300 import evo_attn as E
from memory_efficient_biased_gb300 import evo_seq as Q
from memory_efficient_biased_gb300.autograd import prompt_attention, rotary
from oracle import seq_oracle as O
from tests import seq8_util as C
from tests import seq_util as S

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
NAN8 = 0x7f


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ rotary
def check_rotated(x, got, pos, f, interleaved, factor, inverse=False):
    """Per element: u |y| (rounding), and factor (|x1| + |x2|) 2^-21 for the angle (its conversion to 32
    bits 2^-23 of a radian), sincospif (2^-22) and three roundings in 32 bits; what is not turned is equal."""
    u, tiny = S.U[x.dtype], S.TINY[x.dtype]
    x, got, R = S.f64(x), S.f64(got), 2 * len(f)
    y = O.rotate(x, pos, f, interleaved, factor, inverse)
    near = np.abs(x)
    one, two = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    near[..., one] = near[..., two] = near[..., one] + near[..., two]
    S.assert_close(got[..., :R], y[..., :R], (u * np.abs(y) + factor * 2.0 ** -21 * near)[..., :R] + tiny, "turned")
    np.testing.assert_array_equal(got[..., R:], x[..., R:])


ROTARY = [(1, 1, 1, 64, 64), (3, 8, 2, 128, 128), (70, 4, 4, 72, 72), (33, 5, 0, 128, 96), (257, 32, 8, 128, 64), (19, 3, 7, 40, 10),
          (7, 2, 1, 8, 2), (41, 12, 3, 104, 52), (600, 9, 2, 80, 24)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROTARY)
def test_rotary(T, Hq, Hk, D, R, interleaved, dtype):
    rng = np.random.default_rng(T * R)
    q, k = S.normal(rng, T, Hq, D, dtype=dtype), S.normal(rng, T, Hk, D, dtype=dtype) if Hk else None
    pos = rng.integers(-50, 5000, T).astype(np.int32)
    f, _ = Q.rotary_frequencies(R)
    how = dict(interleaved=interleaved, factor=1.25)
    dq, dk = q.cuda(), None if k is None else k.cuda()
    qo, ko = Q.evo_rotary(dq, dk, i32(pos), f.cuda(), **how)
    check_rotated(q, qo, pos, f.numpy(), interleaved, 1.25)
    if k is None:
        assert ko is None
    else:
        check_rotated(k, ko, pos, f.numpy(), interleaved, 1.25)
    back, _ = Q.evo_rotary(dq, dk, i32(pos), f.cuda(), inverse=True, **how)
    check_rotated(q, back, pos, f.numpy(), interleaved, 1.25, True)
    # in place, the same bytes
    Q.evo_rotary(dq, dk, i32(pos), f.cuda(), dq, dk, **how)
    assert torch.equal(dq, qo) and (k is None or torch.equal(dk, ko))


def test_rotary_far_positions():
    """Positions over the whole of 32 bits: the angle is position · inv_freq to 2^-52 of the turns in it
    (2^31 positions: 2^-21 of a turn at the fastest pair, in the oracle's own product as much)."""
    rng = np.random.default_rng(0)
    q = S.normal(rng, 64, 2, 64, dtype=BF)
    f = Q.rotary_frequencies(64, 500000.0, scaling="parts", stretch=8.0, trained=8192)[0]
    for pos in (rng.integers(0, 1 << 20, 64), rng.integers(-(1 << 31), 1 << 31, 64)):
        out, _ = Q.evo_rotary(q.cuda(), None, i32(pos), f.cuda())
        x, R = S.f64(q), 64
        # the oracle's angle again in integers: 2^64 turns as Python numbers, of the exact double
        from fractions import Fraction
        two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
        a = np.array([[float((int(p) * Fraction(float(w)) / two_pi) % 1) for w in f] for p in pos]) * 2 * np.pi
        z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * a)[:, None]
        y = np.concatenate([z.real, z.imag], -1)
        near = np.tile(np.abs(x[..., :32]) + np.abs(x[..., 32:]), 2)
        turns = np.abs(np.asarray(pos, np.float64))[:, None] * 2.0 ** -52 * 6.3 * np.tile(f.numpy(), 2)[None]
        S.assert_close(S.f64(out), y, 2.0 ** -8 * np.abs(y) + (2.0 ** -21 + turns[:, None]) * near, "far")


def test_rotary_strided_streams_and_graph():
    rng = np.random.default_rng(1)
    T, Hq, Hk, D = 50, 6, 2, 64
    qkv = S.normal(rng, T, (Hq + 2 * Hk) * D, dtype=BF).cuda()
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    pos, f = i32(np.arange(T)), Q.rotary_frequencies(32)[0].cuda()
    want = Q.evo_rotary(q.contiguous(), k.contiguous(), pos, f)
    for x, y in zip(Q.evo_rotary(q, k, pos, f), want):
        assert torch.equal(x, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = Q.evo_rotary(q, k, pos, f, stream=st)
    st.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    tail = qkv[:, (Hq + Hk) * D:].clone()
    keep = qkv.clone()
    qo, ko = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.evo_rotary(q, k, pos, f, qo, ko)
    pos.add_(5)
    g.replay()
    assert torch.equal(qo, Q.evo_rotary(q, k, pos, f)[0]) and not torch.equal(qo, want[0])
    pos.sub_(5)
    Q.evo_rotary(q, k, pos, f, q, k)  # in place, in the projection
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, (Hq + Hk) * D:], tail)
    assert torch.equal(keep[:, (Hq + Hk) * D:], tail)
    assert Q.evo_rotary(q[:0], k[:0], pos[:0], f)[0].shape == (0, Hq, D)


def test_rotary_refusals():
    q, k = torch.zeros(4, 2, 64, dtype=BF, device="cuda"), torch.zeros(4, 1, 64, dtype=BF, device="cuda")
    pos, f = i32([0, 1, 2, 3]), torch.ones(32, dtype=torch.float64, device="cuda")
    for bad in (dict(k=k.half()), dict(k=k[:3]), dict(k=k[..., :32]), dict(positions=pos.long()), dict(positions=pos[:3]),
                dict(inv_freq=f.float()), dict(inv_freq=torch.ones(33, dtype=torch.float64, device="cuda")),
                dict(inv_freq=f[:0]), dict(inv_freq=f.view(4, 8)), dict(factor=float("nan")), dict(factor=0.0),
                dict(q_out=q[:3]), dict(k=None, k_out=k), dict(q=q.transpose(1, 2)), dict(positions=pos.cpu()),
                dict(positions=torch.zeros(8, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises(ValueError):
            Q.evo_rotary(**{**dict(q=q, k=k, positions=pos, inv_freq=f), **bad})
    with pytest.raises(E.EvoAttnError):  # an output over another tensor
        Q.evo_rotary(q, k, pos, f, q_out=torch.empty_like(q), k_out=q[:, :1].as_strided((4, 1, 64), (64, 64, 1)))


def test_rotary_gradient():
    """Against the inverse turn and differences of the operator itself (fp16: a step of 2^-3 moves an output by
    eighths, their roundings by 2^-11 of it)."""
    rng = np.random.default_rng(2)
    T, f = 37, Q.rotary_frequencies(48)[0]
    q, k, gq, gk = (S.normal(rng, T, h, 64, dtype=FP).cuda() for h in (3, 2, 3, 2))
    pos = i32(rng.integers(0, 3000, T))
    for interleaved in (False, True):
        lq, lk = q.clone().requires_grad_(), k.clone().requires_grad_()
        a, b = rotary(lq, lk, pos, f.cuda(), interleaved=interleaved, factor=0.75)
        torch.autograd.backward([a, b], [gq, gk])
        check_rotated(gq, lq.grad, pos.cpu().numpy(), f.numpy(), interleaved, 0.75, True)
        check_rotated(gk, lk.grad, pos.cpu().numpy(), f.numpy(), interleaved, 0.75, True)
        for _ in range(8):
            t, h, d = rng.integers(0, T), rng.integers(0, 3), rng.integers(0, 64)
            up, dn = q.clone(), q.clone()
            up[t, h, d] += 0.125
            dn[t, h, d] -= 0.125
            two = [S.f64(Q.evo_rotary(x, None, pos, f.cuda(), interleaved=interleaved, factor=0.75)[0])[t, h] for x in (up, dn)]
            step = float(up[t, h, d].double() - dn[t, h, d].double())
            got, want = float(lq.grad[t, h, d]), float(((two[0] - two[1]) * S.f64(gq)[t, h]).sum() / step)
            err = (2.0 ** -11 * (np.abs(two[0]) + np.abs(two[1])) * np.abs(S.f64(gq)[t, h]) / step).sum()
            assert abs(got - want) <= err + 2.0 ** -11 * abs(got) + 1e-4
    lq = q.clone().requires_grad_()
    a, none = rotary(lq, None, pos, f.cuda())
    assert none is None
    a.backward(gq)
    check_rotated(gq, lq.grad, pos.cpu().numpy(), f.numpy(), False, 1.0, True)
    # only one of the outputs used
    lq, lk = q.clone().requires_grad_(), k.clone().requires_grad_()
    rotary(lq, lk, pos, f.cuda())[1].backward(gk)
    assert torch.all(lq.grad == 0)
    check_rotated(gk, lk.grad, pos.cpu().numpy(), f.numpy(), False, 1.0, True)


# ------------------------------------------------------------------------------ append and read
def expect_append(cache, state, k, v, chunks, ends):
    """Runs the oracle's append over state[b] = (kcodes [places, H, D], kscales [blocks, H], v...)."""
    a = 0
    for b, (n, end) in enumerate(zip(chunks, ends)):
        for codes, scales, x in ((state[b][0], state[b][1], k), (state[b][2], state[b][3], v)):
            rows = S.f64(x[a:a + n])[max(0, n - end):]
            for h in range(codes.shape[1]):
                c, s = codes[:, h].copy(), scales[:, h].copy()
                O.append8(c, s, rows[:, h], end - len(rows), cache.block)
                codes[:, h], scales[:, h] = c, s
        a += n


def fresh_state(cache, H, D):
    n = cache.table.shape[1] * cache.page
    return [[np.full((n, H, D), np.nan), np.full((n // cache.block, H), -7.0), np.full((n, H, D), np.nan),
             np.full((n // cache.block, H), -7.0)] for _ in range(cache.table.shape[0])]


def assert_holds(cache, state):
    """Every page of the tables holds what the oracle's state says, and no other page anything."""
    table = cache.table.cpu().numpy()
    for (pages, scales), at in (((cache.k, cache.ks), 0), ((cache.v, cache.vs), 2)):
        codes = C.value_of(pages, torch.ones_like(scales))
        s = scales.double().cpu().numpy()
        for b, row in enumerate(table):
            np.testing.assert_array_equal(np.concatenate(list(codes[row])), state[b][at], f"codes of sequence {b}")
            np.testing.assert_array_equal(np.concatenate([x.T for x in s[row]]), state[b][at + 1], f"scales of sequence {b}")
        rest = np.setdiff1d(np.arange(len(codes)), table)
        assert np.all(np.isnan(codes[rest])) and np.all(s[rest] == -7.0)


APPENDS = [([1], [1], 16, 16, 1, 64), ([5, 1, 0, 17], [5, 40, 9, 17], 16, 16, 2, 128), ([130, 3], [300, 64], 64, 32, 3, 80),
           ([33, 200, 1], [33, 300, 129], 128, 128, 2, 48), ([64, 15, 16, 1], [64, 31, 16, 17], 32, 16, 8, 16),
           ([300], [700], 384, 128, 1, 112), ([7, 1], [1000, 63], 64, 64, 5, 128)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("chunks,ctx,page,block,H,D", APPENDS)
def test_append8(chunks, ctx, page, block, H, D, dtype):
    """First what was there, then the chunk behind it, its tokens of very different sizes."""
    rng = np.random.default_rng(sum(ctx) + D)
    cache = C.Cache(rng, ctx, page, block, H, D)
    state = fresh_state(cache, H, D)
    for sizes, ends in (([e - n for n, e in zip(chunks, ctx)], [e - n for n, e in zip(chunks, ctx)]), (chunks, ctx)):
        T = sum(sizes)
        k, v = (S.normal(rng, T, H, D, dtype=torch.float32) * torch.from_numpy(np.exp(rng.standard_normal((T, H, 1)) * 1.5)).float()
                for _ in "kv")
        k, v = k.to(dtype), v.to(dtype)
        Q.evo_cache8_append(k.cuda(), v.cuda(), S.offsets(sizes).cuda(), i32(ends), *cache.args(), cache.table)
        expect_append(cache, state, k, v, sizes, ends)
        assert_holds(cache, state)
    # and out of it: whole sequences, and the newest tokens of them
    for back in (ctx, [min(3, x) for x in ctx]):
        for out in (BF, FP):
            ko, vo = Q.evo_cache8_read(*cache.args(), S.offsets(back).cuda(), i32(ctx), cache.table, sum(back), out)
            a = 0
            for b, n in enumerate(back):
                want = [torch.from_numpy(x[ctx[b] - n:ctx[b]]).to(out).double().numpy() for x in cache.rows(b, ctx[b])]
                np.testing.assert_array_equal(S.f64(ko[a:a + n]), want[0])
                np.testing.assert_array_equal(S.f64(vo[a:a + n]), want[1])
                a += n
    assert E.evo_attn_device_status() == 0


def test_append8_token_by_token():
    """Tokens that grow and shrink, one at a time, over blocks of 16 and of 64."""
    rng = np.random.default_rng(7)
    for page, block in ((16, 16), (64, 64)):
        cache = C.Cache(rng, [90, 90], page, block, 2, 64)
        state = fresh_state(cache, 2, 64)
        for i in range(90):
            size = 2.0 ** rng.integers(-6, 7)
            k, v = (S.normal(rng, 2, 2, 64, dtype=BF, sigma=size) for _ in "kv")
            Q.evo_cache8_append(k.cuda(), v.cuda(), i32([0, 1, 2]), i32([i + 1, i + 1]), *cache.args(), cache.table)
            expect_append(cache, state, k, v, [1, 1], [i + 1, i + 1])
        assert_holds(cache, state)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_append8_extremes(dtype):
    """Zeros, the smallest and largest numbers, infinities and NaN; reading saturates."""
    rng = np.random.default_rng(8)
    big = torch.finfo(dtype).max
    k = torch.zeros(64, 1, 16, dtype=dtype)
    k[16:32] = S.normal(rng, 16, 1, 16, dtype=dtype, sigma=1e-3)
    k[16, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    k[32:48] = big
    k[33] = -big
    k[48:64] = torch.finfo(dtype).tiny
    k[50:52] = float("nan")
    v = k.flip(0).contiguous()
    cache = C.Cache(rng, [64], 16, 16, 1, 16)
    state = fresh_state(cache, 1, 16)
    Q.evo_cache8_append(k.cuda(), v.cuda(), i32([0, 64]), i32([64]), *cache.args(), cache.table)
    expect_append(cache, state, k, v, [64], [64])
    assert_holds(cache, state)
    ko, vo = Q.evo_cache8_read(*cache.args(), i32([0, 64]), i32([64]), cache.table, 64, dtype)
    assert torch.all(ko[32] == big) and torch.all(ko[33] == -big) and torch.all(ko[:16] == 0)
    assert torch.all(torch.isnan(ko[16, 0, :3])) and torch.all(torch.isnan(ko[50:52])) and torch.all(torch.isfinite(ko[17:50]))
    assert torch.equal(torch.nan_to_num(vo, nan=7.0), torch.nan_to_num(ko.flip(0), nan=7.0))


def test_append8_behind_scales_of_others():
    """Tokens behind some whose scale is 0, and they 0 with it whatever their codes; whose scale is no power of two."""
    rng = np.random.default_rng(27)
    for block, old in ((16, 0.0), (64, 0.0), (64, 1.5 * 2.0 ** -12), (32, 1.25 * 2.0 ** 9)):
        cache = C.Cache(rng, [60], 64, block, 2, 64)
        cache.fill(0, *(rng.standard_normal((21, 2, 64)) for _ in "kv"))
        for s in (cache.ks, cache.vs):
            s[s > 0] = old
        page = int(cache.table[0, 0])
        state = fresh_state(cache, 2, 64)
        for at, (pages, scales) in ((0, (cache.k, cache.ks)), (2, (cache.v, cache.vs))):
            state[0][at][:] = C.value_of(pages, torch.ones_like(scales))[page]
            state[0][at + 1][:] = scales[page].double().cpu().numpy().T
        k, v = (S.normal(rng, 9, 2, 64, dtype=BF) for _ in "kv")
        Q.evo_cache8_append(k.cuda(), v.cuda(), i32([0, 9]), i32([30]), *cache.args(), cache.table)
        if old == 0.0:
            expect_append(cache, state, k, v, [9], [30])
            assert_holds(cache, state)
        else:
            got, want = cache.rows(0, 30), [np.concatenate([state[0][at][:21] * old, S.f64(x)]) for at, x in ((0, k), (2, v))]
            for x, y, s in zip(got, want, (cache.ks, cache.vs)):
                # a rounding to three bits, after one in 32 bits that may move it over a border
                least = float(s[page].max()) * 2.0 ** -10
                assert np.all(np.abs(x - y) <= np.abs(y) * (2.0 ** -4 + 2.0 ** -20) + least)


def test_append8_strided_pages_and_rows():
    rng = np.random.default_rng(9)
    cache = C.Cache(rng, [100, 30], 32, 32, 2, 64, interleaved=True)
    state = fresh_state(cache, 2, 64)
    kv = S.normal(rng, 130, 4 * 64, dtype=FP)
    k, v = kv[:, :128].view(130, 2, 64), kv[:, 128:].view(130, 2, 64)
    d = kv.cuda()
    Q.evo_cache8_append(d[:, :128].view(130, 2, 64), d[:, 128:].view(130, 2, 64), i32([0, 100, 130]), i32([100, 30]),
                        *cache.args(), cache.table)
    expect_append(cache, state, k, v, [100, 30], [100, 30])
    assert_holds(cache, state)
    out = torch.full((140, 4 * 64), 7.0, dtype=FP, device="cuda")
    ko, vo = out[:, :128].view(140, 2, 64), out[:, 128:].view(140, 2, 64)
    Q.evo_cache8_read(*cache.args(), i32([5, 15, 35]), i32([100, 30]), cache.table, 140, FP, ko, vo)
    assert torch.all(out[:5] == 7) and torch.all(out[35:] == 7)
    for b, (lo, n, end) in enumerate(((5, 10, 100), (15, 20, 30))):
        for x, want in zip((ko, vo), cache.rows(b, end)):
            np.testing.assert_array_equal(S.f64(x[lo:lo + n]), torch.from_numpy(want[end - n:]).to(FP).double().numpy())


def test_append8_more_tokens_than_length_and_rows_outside():
    """A new token at a negative position is not written; rows in no sequence are not read."""
    rng = np.random.default_rng(10)
    cache = C.Cache(rng, [40, 40], 16, 16, 1, 32)
    state = fresh_state(cache, 1, 32)
    k, v = (S.normal(rng, 40, 1, 32, dtype=BF) for _ in "kv")
    k[:3] = v[36:] = float("nan")
    Q.evo_cache8_append(k.cuda(), v.cuda(), i32([3, 23, 36]), i32([8, 13]), *cache.args(), cache.table)
    expect_append(cache, state, k[3:36], v[3:36], [20, 13], [8, 13])
    assert_holds(cache, state)
    ko, _ = Q.evo_cache8_read(*cache.args(), i32([0, 12, 15]), i32([8, 13]), cache.table, 15, BF)
    assert torch.all(ko[:4] == 0)
    np.testing.assert_array_equal(S.f64(ko[4:12]), cache.rows(0, 8)[0])


def test_append8_many_sequences():
    """More sequences than three rounds of the search for a block's tell apart, most of them short, some empty."""
    rng = np.random.default_rng(12)
    n = 1500
    had, new = rng.integers(0, 20, n), rng.integers(0, 4, n)
    new[[0, 700, 1499]] = 0, 60, 33
    ends = [int(x) for x in had + new]
    cache = C.Cache(rng, [max(ends)] * n, 16, 16, 1, 16)
    state = fresh_state(cache, 1, 16)
    for sizes, lens in (([int(x) for x in had], [int(x) for x in had]), ([int(x) for x in new], ends)):
        T = sum(sizes)
        k, v = (S.normal(rng, T, 1, 16, dtype=BF, sigma=float(s)) for s in (1.0, 3.0))
        Q.evo_cache8_append(k.cuda(), v.cuda(), S.offsets(sizes).cuda(), i32(lens), *cache.args(), cache.table)
        expect_append(cache, state, k, v, sizes, lens)
    assert_holds(cache, state)
    ko, vo = Q.evo_cache8_read(*cache.args(), S.offsets(ends).cuda(), i32(ends), cache.table, sum(ends), BF)
    a = 0
    for b, e in enumerate(ends):
        s = np.repeat(state[b][1], 16, 0)[:e, :, None]
        np.testing.assert_array_equal(S.f64(ko[a:a + e]), state[b][0][:e] * s)
        a += e
    q = S.normal(rng, n, 2, 16, dtype=BF)
    out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), i32(np.arange(n + 1)), i32(ends), cache.table)
    for b in list(range(0, n, 37)) + [700, 1499]:
        rows = cache.rows(b, ends[b])
        C.check_attention(S.f64(q[b:b + 1]), *rows, S.f64(out[b:b + 1]), S.f64(lse[:, b:b + 1]), 0.25, BF, f"sequence {b}")
    assert E.evo_attn_device_status() == 0


def test_offsets_out_of_order_with_more_rows_than_tokens():
    """Recorded; nothing is written that is not a row of the call or a page of the tables."""
    rng = np.random.default_rng(13)
    for Hq in (2, 8, 64):  # the three ways of the attention
        cache = C.Cache(rng, [60] * 5, 16, 16, 1, 64)
        k, v, q = (S.normal(rng, 60, h, 64, dtype=BF).cuda() for h in (1, 1, Hq))
        cu, lens = i32([0, 60, 0, 60, 0, 60]), i32([60] * 5)
        for call in (lambda s: Q.evo_cache8_append(k, v, cu, lens, *cache.args(), cache.table, status=s),
                     lambda s: Q.evo_cache8_read(*cache.args(), cu, lens, cache.table, 60, BF, status=s),
                     lambda s: Q.evo_paged8_fwd(q, *cache.args(), cu, lens, cache.table, status=s)):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(status)
            assert int(status) == 13
        rest = np.setdiff1d(np.arange(cache.k.shape[0]), cache.table.cpu().numpy())
        assert torch.all(cache.k.view(torch.uint8)[torch.from_numpy(rest).cuda()] == NAN8)
    assert E.evo_attn_device_status() == 0


def test_bad_indices_are_recorded_and_leave_the_rest():
    rng = np.random.default_rng(11)
    for what in ("offset", "length", "long", "page"):
        cache = C.Cache(rng, [40, 40, 40], 16, 16, 2, 64)
        k, v, q = (S.normal(rng, 60, h, 64, dtype=BF).cuda() for h in (2, 2, 4))
        cu, lens, table = [0, 20, 40, 60], [40, 40, 40], cache.table.clone()
        if what == "offset":
            cu[2] = 61
        elif what == "length":
            lens[1] = -3
        elif what == "long":
            lens[1] = 49
        else:
            table[1, 1:] = i32([-1, table.max() + 50])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.evo_cache8_append(k, v, i32(cu), i32(lens), *cache.args(), table, status=status)
        assert int(status) == 13, what
        state = fresh_state(cache, 2, 64)
        expect_append(cache, state, k[:20], v[:20], [20], [40])
        if what != "offset":  # (the third sequence's own offset is bad too there)
            a, b = state[:2], state[2:]
            expect_append(cache, b, k[40:], v[40:], [20], [40])
        if what == "page":
            expect_append(cache, state[1:], k[20:40], v[20:40], [20], [40])
            for x in (0, 2):  # places 16 and on have no page
                state[1][x][16:] = np.nan
                state[1][x + 1][1:] = -7.0
        assert_holds(cache, state)
        status.zero_()
        Q.evo_cache8_read(*cache.args(), i32(cu), i32(lens), table, 60, BF, status=status)
        assert int(status) == 13, what
        status.zero_()
        # (tokens 0 .. 19 are not there: as a cache holds what was appended)
        cache.fill(0, *(rng.standard_normal((40, 2, 64)) for _ in "kv"))
        out, lse = Q.evo_paged8_fwd(q, *cache.args(), i32(cu), i32(lens), table, status=status)
        assert int(status) == 13, what
        C.check_attention(S.f64(q[:20]), *cache.rows(0, 40), S.f64(out[:20]), S.f64(lse[:, :20]), 64 ** -0.5, BF, what)
    assert E.evo_attn_device_status() == 0


# ------------------------------------------------------------------------------ attention
def filled(rng, ctx, page, block, Hk, D, spread=0.7, **kw):
    """A cache of sequences of ctx[b] tokens whose tokens differ in size (and so blocks in scale)."""
    cache = C.Cache(rng, ctx, page, block, Hk, D, **kw)
    for b, n in enumerate(ctx):
        cache.fill(b, *(rng.standard_normal((n, Hk, D)) * np.exp(rng.standard_normal((n // 9 + 1, Hk, 1)) * spread).repeat(9, 0)[:n]
                        for _ in "kv"))
    return cache


def check_paged(cache, q, chunks, ctx, out, lse, scale, dtype, skip=(), **kw):
    a = 0
    for b, (n, end) in enumerate(zip(chunks, ctx)):
        if n and b not in skip:
            C.check_attention(S.f64(q[a:a + n]), *cache.rows(b, end), S.f64(out[a:a + n]), S.f64(lse[:, a:a + n]), scale, dtype,
                              f"sequence {b}", **kw)
        a += n


PAGED = [([1], [1], 1, 1, 64, 16, 16), ([1], [777], 8, 2, 128, 16, 16), ([1, 1, 1, 1], [40, 1, 129, 1000], 4, 4, 128, 64, 32),
         ([1, 0, 1], [513, 9, 64], 16, 1, 128, 128, 128), ([3, 1, 2], [300, 256, 2], 5, 1, 80, 32, 16),
         ([17, 5], [17, 400], 6, 2, 96, 16, 16), ([130, 1, 64], [130, 700, 333], 4, 2, 128, 64, 64),
         ([200], [900], 8, 1, 64, 384, 128), ([1, 40], [260, 41], 128, 1, 64, 16, 16), ([2, 1], [99, 130], 24, 1, 48, 32, 32),
         ([1] * 40, [7 + 31 * i % 400 for i in range(40)], 8, 2, 16, 16, 16), ([5, 9], [600, 1300], 3, 3, 112, 1024, 64),
         ([8, 5, 8], [3000, 900, 2500], 8, 2, 128, 64, 16), ([9, 8], [1700, 60], 8, 2, 64, 32, 32)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("chunks,ctx,Hq,Hk,D,page,block", PAGED)
def test_paged8(chunks, ctx, Hq, Hk, D, page, block, dtype):
    rng = np.random.default_rng(sum(ctx))
    cache = filled(rng, ctx, page, block, Hk, D)
    q = S.normal(rng, sum(chunks), Hq, D, dtype=dtype, sigma=1.3)
    args = q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table
    out, lse = Q.evo_paged8_fwd(*args)
    check_paged(cache, q, chunks, ctx, out, lse, D ** -0.5, dtype)
    again = Q.evo_paged8_fwd(*args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert E.evo_attn_device_status() == 0


def test_paged8_long_context():
    """One context over every SM, its pieces joined; few rows and a chunk of them."""
    rng = np.random.default_rng(20)
    for chunks, ctx in (([1, 2], [20011, 5000]), ([70, 1], [9001, 4100])):
        cache = filled(rng, ctx, 64, 16, 2, 64)
        q = S.normal(rng, sum(chunks), 8, 64, dtype=BF, sigma=1.3)
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table)
        check_paged(cache, q, chunks, ctx, out, lse, 0.125, BF)


def test_paged8_given_scales_and_scale():
    """Scales that are no powers of two, blocks whose scales lie far apart, a softmax scale."""
    rng = np.random.default_rng(21)
    for chunks, ctx, dtype in (([1, 1], [300, 77], FP), ([60, 3], [300, 77], FP), ([60], [200], BF)):
        cache = C.Cache(rng, ctx, 32, 32, 2, 64)
        for b, n in enumerate(ctx):
            own = lambda rows: np.abs(rows).max((0, 2)) / 448 * rng.uniform(1.0, 2.0, 2)  # noqa: E731
            cache.fill(b, *(rng.standard_normal((n, 2, 64)) * 10.0 ** rng.integers(-2, 2, (n // 32 + 1, 2, 1)).repeat(32, 0)[:n]
                            for _ in "kv"), scale=lambda rows: np.float32(own(rows)).astype(np.float64))
        q = S.normal(rng, sum(chunks), 4, 64, dtype=dtype)
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table, scale=0.05)
        vmax = 448 * float(cache.vs.max())
        check_paged(cache, q, chunks, ctx, out, lse, float(np.float32(0.05)), dtype, vmax=vmax)


@pytest.mark.parametrize("chunks,ctx", [([1, 2], [300, 77]), ([1], [3000]), ([60, 3], [300, 77]), ([300], [301])])
def test_paged8_scales_of_zero(chunks, ctx):
    """Blocks of zeros with a scale of 0, as others may write them, and as an append leaves them, 2^-64: their keys (the first of them
    with large scores against the others') have weight, their values none.  The blocks of keys that are zero the same."""
    rng = np.random.default_rng(26)
    for zero in (0.0, 2.0 ** -64):
        cache = C.Cache(rng, ctx, 32, 32, 2, 64)
        for b, n in enumerate(ctx):
            k, v = (rng.standard_normal((n, 2, 64)) for _ in "kv")
            v[:32, 0] = v[-40:, 1] = k[32:64, 1] = 0.0
            k[:32] *= 3.0
            cache.fill(b, k, v)
        for s in (cache.ks, cache.vs):
            s[s == 2.0 ** -64] = zero
        q = S.normal(rng, sum(chunks), 4, 64, dtype=BF)
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table)
        check_paged(cache, q, chunks, ctx, out, lse, 0.125, BF)


def test_paged8_rising_scores():
    """A maximum that moves far, more than once, in some rows only."""
    rng = np.random.default_rng(22)
    for chunks, ctx in (([1], [900]), ([150], [900])):
        cache = C.Cache(rng, ctx, 64, 64, 1, 64)
        k = rng.standard_normal((900, 1, 64)) * (1 + np.arange(900) / 150)[:, None, None]
        cache.fill(0, k, rng.standard_normal((900, 1, 64)) * np.exp(-np.arange(900) / 100)[:, None, None])
        q = S.normal(rng, chunks[0], 2, 64, dtype=BF)
        q[:, 0] *= 4
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table)
        check_paged(cache, q, chunks, ctx, out, lse, 0.125, BF)


def test_paged8_unseen_values_do_not_spread():
    """Codes that are NaN, and scales of any kind, behind a sequence's end; NaN in later tokens of the same chunk."""
    rng = np.random.default_rng(23)
    for chunks, ctx, Hq, Hk in (([1, 1], [70, 33], 4, 2), ([50, 20], [70, 33], 4, 2), ([9, 33], [9, 161], 8, 1)):
        cache = filled(rng, ctx, 64, 16, Hk, 128)
        clean = [cache.rows(b, n) for b, n in enumerate(ctx)]
        for s in (cache.ks, cache.vs):
            s[s == -7.0] = float("nan")
        # the last token of the first sequence: only its own row sees it
        at = ctx[0] - 1
        p = int(cache.table[0, at // 64])
        cache.k.view(torch.uint8)[p, at % 64, :, 5] = NAN8
        cache.v.view(torch.uint8)[p, at % 64, :, 9] = NAN8 | 128
        q = S.normal(rng, sum(chunks), Hq, 128, dtype=BF)
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table)
        a = 0
        for b, (n, end) in enumerate(zip(chunks, ctx)):
            rows = n - (b == 0)
            k, v = clean[b]
            C.check_attention(S.f64(q[a:a + rows]), k[:end - n + rows], v[:end - n + rows], S.f64(out[a:a + rows]),
                              S.f64(lse[:, a:a + rows]), 128 ** -0.5, BF, f"sequence {b}")
            a += n
        assert torch.all(torch.isnan(out[chunks[0] - 1])) and torch.all(torch.isnan(lse[:, chunks[0] - 1]))
        # NaN in a value alone: in that feature alone
        cache.k.view(torch.uint8)[p, at % 64, :, 5] = 0
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table)
        last = out[chunks[0] - 1].float()
        assert torch.all(torch.isnan(last[:, 9])) and torch.all(torch.isfinite(last[:, :9])) and torch.all(torch.isfinite(last[:, 10:]))


def test_paged8_rows_that_see_nothing():
    """More new tokens than the length, a length of zero, rows outside every sequence."""
    rng = np.random.default_rng(24)
    for chunks, ctx in (([6, 3, 1], [4, 0, 50]), ([200, 40, 1], [90, 0, 50])):
        cache = filled(rng, [max(1, x) for x in ctx], 16, 16, 2, 64)
        T = sum(chunks) + 7
        q = S.normal(rng, T, 4, 64, dtype=FP).cuda()
        out, lse = torch.full_like(q, 7.0), torch.full((4, T), 7.0, device="cuda")
        Q.evo_paged8_fwd(q, *cache.args(), (S.offsets(chunks) + 3).cuda(), i32(ctx), cache.table, out, lse)
        a = 3
        assert torch.all(out[:3] == 7) and torch.all(out[T - 4:] == 7) and torch.all(lse[:, :3] == 7) and torch.all(lse[:, T - 4:] == 7)
        for b, (n, end) in enumerate(zip(chunks, ctx)):
            none = max(0, n - end)
            assert torch.all(out[a:a + none] == 0) and torch.all(lse[:, a:a + none] == -float("inf"))
            if n > none:
                C.check_attention(S.f64(q[a + none:a + n]), *cache.rows(b, end), S.f64(out[a + none:a + n]),
                                  S.f64(lse[:, a + none:a + n]), 0.125, FP, f"sequence {b}")
            a += n
    assert E.evo_attn_device_status() == 0


def test_paged8_strided_streams_graphs_and_workspaces():
    rng = np.random.default_rng(25)
    for chunks, ctx in (([1, 1, 1], [200, 3000, 41]), ([100, 1, 30], [200, 3000, 41])):
        T, Hq, Hk, D = sum(chunks), 4, 2, 64
        cache = filled(rng, ctx, 32, 16, Hk, D, interleaved=True)
        wide = S.normal(rng, T, 2 * Hq * D, dtype=BF).cuda()
        q = wide[:, :Hq * D].view(T, Hq, D)
        rest = *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table
        want, z = Q.evo_paged8_fwd(q.contiguous(), *rest)
        check_paged(cache, q.cpu(), chunks, ctx, want, z, D ** -0.5, BF)
        room = torch.zeros(T, 3 * Hq * D, dtype=BF, device="cuda")
        Q.evo_paged8_fwd(q, *rest, out=room[:, Hq * D:2 * Hq * D].view(T, Hq, D))
        assert torch.equal(room[:, Hq * D:2 * Hq * D].reshape(T, Hq, D), want)
        assert torch.all(room[:, :Hq * D] == 0) and torch.all(room[:, 2 * Hq * D:] == 0)
        # two streams at once, each with a workspace of its own
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [Q.evo_paged8_fwd(q, *rest, stream=st) for st in streams for _ in range(3)]
        torch.cuda.synchronize()
        for o, l in got:
            assert torch.equal(o, want) and torch.equal(l, z)
        # captured, and replayed on other queries and a longer context
        out, lse, g = torch.empty_like(want), torch.empty_like(z), torch.cuda.CUDAGraph()
        ws = torch.empty(Q.evo_paged8_fwd_workspace_bytes(T, 3, Hq, Hk, D, cache.k.shape[0], 32, cache.table.shape[1], 16),
                         dtype=torch.uint8, device="cuda")
        lens = i32(ctx)
        with torch.cuda.graph(g):
            Q.evo_paged8_fwd(q, *cache.args(), rest[4], lens, cache.table, out=out, lse=lse, workspace=ws)
        ws.fill_(255)
        wide.mul_(0.5)
        lens.sub_(i32([1, 700, 1]))
        g.replay()
        fresh = Q.evo_paged8_fwd(q, *cache.args(), rest[4], lens, cache.table)
        assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1]) and not torch.equal(out, want)
        with pytest.raises(E.EvoAttnError):
            Q.evo_paged8_fwd(q, *rest, workspace=ws[:1024])


def test_paged8_past_32_bits_of_offset():
    """Pages that lie more than 2^32 elements into the cache, and a stride of them."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    rng = np.random.default_rng(26)
    Hk, D, page, n = 8, 128, 128, 36000  # 2^17 elements a page: 4.7e9
    k, v = (torch.zeros(n, page, Hk, D, dtype=torch.uint8, device="cuda").view(C.E4M3) for _ in "kv")
    cache = C.Cache(rng, [300, 300], page, 64, Hk, D)
    small = cache.k, cache.v, cache.ks, cache.vs
    cache.k, cache.v = k, v
    cache.ks, cache.vs = (torch.ones(n, Hk, 2, device="cuda") for _ in "kv")
    cache.table = i32([[35999, 3, 34000], [0, 33333, 35998]])
    del small
    rows = S.normal(rng, 600, 2 * Hk, D, dtype=BF)
    Q.evo_cache8_append(rows[:, :Hk].contiguous().cuda(), rows[:, Hk:].contiguous().cuda(), i32([0, 300, 600]), i32([300, 300]),
                        *cache.args(), cache.table)
    ko, _ = Q.evo_cache8_read(*cache.args(), i32([0, 300, 600]), i32([300, 300]), cache.table, 600, BF)
    err = np.abs(S.f64(ko) - S.f64(rows[:, :Hk]))
    s = np.abs(S.f64(rows[:, :Hk])).max() / 224
    assert np.all(err <= np.maximum(np.abs(S.f64(rows[:, :Hk])) * 2.0 ** -4, s * 2.0 ** -10))
    table = cache.table.cpu().numpy()
    want = []
    for b in range(2):
        sub = [torch.stack([x[int(p)].view(torch.uint8) for p in table[b]]).view(C.E4M3) for x in (k, v)]
        sc = [torch.stack([x[int(p)] for p in table[b]]) for x in (cache.ks, cache.vs)]
        want.append([C.value_of(x, y).reshape(-1, Hk, D)[:300] for x, y in zip(sub, sc)])
    for chunks in ([1, 1], [40, 30]):
        q = S.normal(rng, sum(chunks), Hk, D, dtype=BF)
        out, lse = Q.evo_paged8_fwd(q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32([300, 300]), cache.table)
        a = 0
        for b, m in enumerate(chunks):
            C.check_attention(S.f64(q[a:a + m]), *want[b], S.f64(out[a:a + m]), S.f64(lse[:, a:a + m]), D ** -0.5, BF)
            a += m


COPIED = [([300], [300], 8, 2, 128, 16, 16), ([200, 0, 260], [700, 33, 260], 16, 2, 64, 64, 32), ([33, 70], [500, 400], 64, 1, 80, 32, 32),
          ([600, 1], [1400, 900], 4, 2, 128, 128, 128), ([180], [1025], 12, 4, 96, 384, 64), ([9], [64], 128, 1, 16, 16, 16),
          ([500], [500], 8, 2, 128, 16, 16), ([300, 0, 301], [700, 33, 400], 16, 2, 112, 64, 32), ([30, 70], [1400, 900], 64, 2, 128, 128, 128)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("chunks,ctx,Hq,Hk,D,page,block", COPIED)
def test_paged8_many_rows(chunks, ctx, Hq, Hk, D, page, block, dtype):
    """More rows a key than two blocks: the codes are widened once, into the workspace; with a
    table too wide for that (places for 2^20 tokens and more), where they are used.  Behind the sequences' ends the pages and scales hold NaN."""
    rng = np.random.default_rng(sum(ctx) + 1)
    cache = filled(rng, ctx, page, block, Hk, D)
    for s in (cache.ks, cache.vs):
        s[s == -7.0] = float("nan")
    q = S.normal(rng, sum(chunks), Hq, D, dtype=dtype, sigma=1.3)
    wide = torch.full((len(ctx), (1 << 28) // (Hk * D * page) + 1), -1, dtype=torch.int32, device="cuda")
    wide[:, :cache.table.shape[1]] = cache.table
    need = [Q.evo_paged8_fwd_workspace_bytes(sum(chunks), len(ctx), Hq, Hk, D, cache.k.shape[0], page, t.shape[1], block)
            for t in (cache.table, wide)]
    copied = sum(chunks) * Hq // Hk > 512 * len(ctx)
    assert (need[0] >= 4 * len(ctx) * max(ctx) * Hk * D if copied else need[0] <= need[1]) and need[1] < 1 << 29
    for table in (cache.table, wide):
        args = q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), table
        out, lse = Q.evo_paged8_fwd(*args)
        check_paged(cache, q, chunks, ctx, out, lse, D ** -0.5, dtype)
        again = Q.evo_paged8_fwd(*args)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert E.evo_attn_device_status() == 0


def test_paged8_many_rows_unseen_bad_and_captured():
    """As above: NaN in later tokens of the chunk, a bad page, strided pages, a captured call replayed on a longer context."""
    rng = np.random.default_rng(28)
    chunks, ctx, Hq, Hk, D = [80, 70], [300, 90], 16, 1, 64
    cache = filled(rng, ctx, 32, 16, Hk, D, interleaved=True)
    clean = [cache.rows(b, n) for b, n in enumerate(ctx)]
    q = S.normal(rng, 150, Hq, D, dtype=BF)
    wide = torch.zeros(150, 2 * Hq * D, dtype=BF, device="cuda")
    wide[:, :Hq * D] = q.cuda().view(150, -1)
    qd, cu, lens = wide[:, :Hq * D].view(150, Hq, D), S.offsets(chunks).cuda(), i32(ctx)
    p = int(cache.table[0, 299 // 32])
    cache.v.view(torch.uint8)[p, 299 % 32, 0, 9] = NAN8
    out, lse = Q.evo_paged8_fwd(qd, *cache.args(), cu, lens, cache.table)
    C.check_attention(S.f64(q[:79]), clean[0][0][:299], clean[0][1][:299], S.f64(out[:79]), S.f64(lse[:, :79]), 0.125, BF)
    C.check_attention(S.f64(q[80:]), *clean[1], S.f64(out[80:]), S.f64(lse[:, 80:]), 0.125, BF)
    last = out[79].float()
    assert torch.all(torch.isnan(last[:, 9])) and torch.all(torch.isfinite(last[:, :9])) and torch.all(torch.isfinite(last[:, 10:]))
    cache.v.view(torch.uint8)[p, 299 % 32, 0, 9] = 0
    table, status = cache.table.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    table[1, 0] = -5
    out, lse = Q.evo_paged8_fwd(qd, *cache.args(), cu, lens, table, status=status)
    assert int(status) == 13
    C.check_attention(S.f64(q[:80]), *cache.rows(0, 300), S.f64(out[:80]), S.f64(lse[:, :80]), 0.125, BF)
    ws = torch.empty(Q.evo_paged8_fwd_workspace_bytes(150, 2, Hq, Hk, D, cache.k.shape[0], 32, cache.table.shape[1], 16),
                     dtype=torch.uint8, device="cuda")
    o, z, g = wide[:, Hq * D:].view(150, Hq, D), torch.empty_like(lse), torch.cuda.CUDAGraph()
    lens.sub_(10)
    with torch.cuda.graph(g):
        Q.evo_paged8_fwd(qd, *cache.args(), cu, lens, cache.table, out=o, lse=z, workspace=ws)
    lens.add_(10)
    ws.fill_(255)
    g.replay()
    check_paged(cache, q, chunks, ctx, o, z, 0.125, BF)
    assert E.evo_attn_device_status() == 0


def test_paged8_gives_up_in_time():
    """The least wait limit: a kernel may give up, says so, and leaves the GPU as it was; the next call is as usual."""
    rng = np.random.default_rng(29)
    ctx = [5000, 3000]
    cache = filled(rng, ctx, 64, 64, 2, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for chunks in ([1, 1], [40, 30]):
        q = S.normal(rng, sum(chunks), 8, 128, dtype=BF)
        args = q.cuda(), *cache.args(), S.offsets(chunks).cuda(), i32(ctx), cache.table
        want = Q.evo_paged8_fwd(*args)
        Q.evo_paged8_fwd(*args, wait_limit_ns=1, status=status)
        assert int(status) in (0, 8)
        status.zero_()
        again = Q.evo_paged8_fwd(*args, wait_limit_ns=10 ** 9, status=status)
        assert int(status) == 0
        for x, y in zip(want, again):
            assert torch.equal(x, y)
        check_paged(cache, q, chunks, ctx, *again, 128 ** -0.5, BF)
    assert E.evo_attn_device_status() == 0


def test_paged8_refusals():
    rng = np.random.default_rng(27)
    cache = filled(rng, [40], 16, 16, 2, 64)
    q, cu, lens = torch.zeros(1, 4, 64, dtype=BF, device="cuda"), i32([0, 1]), i32([40])
    good = dict(q=q, k_pages=cache.k, v_pages=cache.v, k_scales=cache.ks, v_scales=cache.vs, cu_seqlens=cu, seq_lens=lens,
                block_table=cache.table)
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :3]), dict(k_pages=cache.k.view(torch.uint8)),
                dict(v_pages=cache.v[1:]), dict(v_pages=cache.v.view(torch.uint8)), dict(k_scales=cache.ks.double()),
                dict(v_scales=cache.vs[:, :1]), dict(v_scales=cache.vs[..., 0]), dict(seq_lens=lens.long()), dict(seq_lens=i32([1, 2])),
                dict(block_table=cache.table[0]), dict(block_table=cache.table.long()), dict(out=q.half()),
                dict(lse=torch.zeros(4, 2, device="cuda")), dict(scale=0.0), dict(scale=-1.0), dict(k_pages=cache.k.transpose(1, 2)),
                dict(k_pages=cache.k[:1].expand(3, 16, 2, 64)), dict(wait_limit_ns=-1), dict(cu_seqlens=cu.float())):
        with pytest.raises(ValueError):
            Q.evo_paged8_fwd(**{**good, **bad})
    with pytest.raises(E.EvoAttnError):  # a block of 8 tokens
        Q.evo_paged8_fwd(**{**good, "k_scales": torch.ones(cache.k.shape[0], 2, 2, device="cuda"),
                            "v_scales": torch.ones(cache.k.shape[0], 2, 2, device="cuda")})
    with pytest.raises(E.EvoAttnError):  # out over the queries
        Q.evo_paged8_fwd(**good, out=q)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF, FP])
def test_serving_run(dtype):
    """Prompts rotated, appended and attended, then steps of single tokens, as a server runs them; each step
    against the oracle on what the cache holds by then."""
    rng = np.random.default_rng(30)
    Hq, Hk, D, R, lens = 8, 2, 64, 32, [37, 130, 5]
    cache = C.Cache(rng, [n + 8 for n in lens], 32, 16, Hk, D)
    f, factor = Q.rotary_frequencies(R, scaling="parts", stretch=4.0, trained=64)
    ends = [0, 0, 0]
    for step in range(7):
        chunks = lens if step == 0 else ([1, 1, 1] if step != 4 else [1, 0, 3])
        first, ends = ends, [e + n for e, n in zip(ends, chunks)]
        T = sum(chunks)
        qkv = S.normal(rng, T, (Hq + 2 * Hk) * D, dtype=dtype)
        d = qkv.cuda()
        q, k, v = d[:, :Hq * D].view(T, Hq, D), d[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D), d[:, (Hq + Hk) * D:].view(T, Hk, D)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(first, chunks)]).astype(np.int32)
        cu, sl = S.offsets(chunks).cuda(), i32(ends)
        plain = S.f64(q)
        Q.evo_rotary(q, k, i32(pos), f.cuda(), q, k, factor=factor)
        check_rotated(torch.from_numpy(plain).to(dtype), q, pos, f.numpy(), False, factor)
        Q.evo_cache8_append(k, v, cu, sl, *cache.args(), cache.table)
        out, lse = Q.evo_paged8_fwd(q, *cache.args(), cu, sl, cache.table)
        check_paged(cache, q.cpu(), chunks, ends, out, lse, D ** -0.5, dtype)
        # the cache holds the rows to half a step of e4m3 (twice where a block's scale grew behind them)
        ko, vo = Q.evo_cache8_read(*cache.args(), cu, sl, cache.table, T, dtype)
        for got, x in ((ko, k), (vo, v)):
            x = S.f64(x)
            assert np.all(np.abs(S.f64(got) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.abs(x).max() / 224 * 2.0 ** -10))
    assert E.evo_attn_device_status() == 0


def test_captured_step():
    """Rotation, append, attention and read of one step captured once and replayed for token after token, the lengths and
    positions counted up inside; a cache that begins empty."""
    rng = np.random.default_rng(32)
    Hq, Hk, D, B, steps = 8, 2, 128, 3, 40
    caches = [C.Cache(np.random.default_rng(1), [steps] * B, 16, 16, Hk, D) for _ in range(2)]
    f = Q.rotary_frequencies(D)[0].cuda()
    rows = S.normal(rng, steps, B, (Hq + 2 * Hk) * D, dtype=BF).cuda()
    cu = i32([0, 1, 2, 3])

    def step(cache, qkv, lens, pos):
        lens.add_(1)
        q, k, v = qkv[:, :Hq * D].view(B, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(B, Hk, D), qkv[:, (Hq + Hk) * D:].view(B, Hk, D)
        q, k = Q.evo_rotary(q, k, pos, f)
        Q.evo_cache8_append(k, v, cu, lens, *cache.args(), cache.table)
        out = Q.evo_paged8_fwd(q, *cache.args(), cu, lens, cache.table)
        pos.add_(1)
        return (*out, *Q.evo_cache8_read(*cache.args(), cu, lens, cache.table, B, BF))

    one, lens, pos = rows[0].clone(), i32([0] * B), i32([0] * B)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):  # (the extension's first launches are no capture's)
        step(C.Cache(np.random.default_rng(1), [steps] * B, 16, 16, Hk, D), one, i32([0] * B), i32([0] * B))
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(caches[0], one, lens, pos)
    l2, p2 = i32([0] * B), i32([0] * B)
    for i in range(steps):
        one.copy_(rows[i])
        g.replay()
        want = step(caches[1], rows[i], l2, p2)
        for x, y in zip(got, want):
            assert torch.equal(x, y), i
    for x, y in zip(caches[0].args(), caches[1].args()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    q = S.f64(Q.evo_rotary(rows[-1][:, :Hq * D].view(B, Hq, D), None, i32([steps - 1] * B), f)[0])
    for b in range(B):
        C.check_attention(q[b:b + 1], *caches[0].rows(b, steps), S.f64(got[0][b:b + 1]), S.f64(got[1][:, b:b + 1]), D ** -0.5, BF)


def test_training_run():
    """rotary in front of prompt_attention, trained through: gradients of the projections against the oracle's
    chain, within what prompt_attention's own gradients may be off, turned back."""
    rng = np.random.default_rng(31)
    lens, Hq, Hk, D = [90, 33], 4, 2, 64
    T = sum(lens)
    f = Q.rotary_frequencies(D)[0]
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    q, k, v, do = (S.normal(rng, T, h, D, dtype=BF) for h in (Hq, Hk, Hk, Hq))
    lq, lk, lv = (x.cuda().requires_grad_() for x in (q, k, v))
    a, b = rotary(lq, lk, i32(pos), f.cuda())
    a.retain_grad(), b.retain_grad()
    out = prompt_attention(a, b, lv, S.offsets(lens).cuda())
    out.backward(do.cuda())
    at = 0
    for n in lens:
        r = slice(at, at + n)
        S.check_gradients(S.f64(a[r]), S.f64(b[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x.grad[r]) for x in (a, b, lv)], D ** -0.5, BF)
        at += n
    check_rotated(a.grad.cpu(), lq.grad, pos, f.numpy(), False, 1.0, True)
    check_rotated(b.grad.cpu(), lk.grad, pos, f.numpy(), False, 1.0, True)
    # captured: forward and backward of the same leaves inside one graph
    g, grads = torch.cuda.CUDAGraph(), None
    lq2, lk2, lv2 = (x.cuda().requires_grad_() for x in (q, k, v))
    cu, p, w, fr = S.offsets(lens).cuda(), i32(pos), do.cuda(), f.cuda()
    with torch.cuda.graph(g):
        a, b = rotary(lq2, lk2, p, fr)
        grads = torch.autograd.grad(prompt_attention(a, b, lv2, cu), (lq2, lk2, lv2), w)
    g.replay()
    for x, y in zip(grads, (lq, lk, lv)):
        assert torch.equal(x, y.grad)
