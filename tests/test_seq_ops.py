"""GPU: the causal-sequence operators against the fp64 oracle, with bounds derived from
their roundings (tests/seq_util.py): packed prompts and their gradients, chunks and
single tokens over a paged cache, the sums of their weights, eviction, and a run of them
together; odd sizes, rows that see nothing, NaN and infinities in unseen places, strided
rows and pages, bad offsets, lengths and pages, streams and captured graphs."""
import numpy as np
import pytest
import torch

from memory_efficient_biased_gb300 import evo_attn as E
from memory_efficient_biased_gb300 import evo_seq as Q
from memory_efficient_biased_gb300.autograd import prompt_attention
from oracle import seq_oracle as O
from tests import seq_util as S

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def prompt_inputs(lens, Hq, Hk, D, dtype, seed=0, extra=0):
    rng = np.random.default_rng(seed)
    T = sum(lens) + extra
    q, do = S.normal(rng, T, Hq, D, dtype=dtype, sigma=1.5), S.normal(rng, T, Hq, D, dtype=dtype)
    return q, S.normal(rng, T, Hk, D, dtype=dtype), S.normal(rng, T, Hk, D, dtype=dtype), do, S.offsets(lens)


def check_prompt(q, k, v, lens, out, lse, scale, dtype, begin=0, skip=()):
    a = begin
    for b, n in enumerate(lens):
        if n and b not in skip:
            S.check_forward(S.f64(q[a:a + n]), S.f64(k[a:a + n]), S.f64(v[a:a + n]), S.f64(out[a:a + n]),
                            S.f64(lse[:, a:a + n]), scale, dtype, f"sequence {b}")
        a += n


PROMPTS = [([1], 1, 1, 64), ([5, 1, 0, 17], 4, 2, 64), ([128, 129, 127], 2, 2, 128), ([300], 8, 1, 128),
           ([40, 333, 0, 1, 64], 6, 2, 96), ([257], 5, 1, 72), ([700, 90], 3, 1, 128), ([64, 65], 12, 4, 8),
           ([513], 2, 1, 40), ([1030], 4, 4, 128), ([200, 31], 128, 1, 64)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,Hq,Hk,D", PROMPTS)
def test_prompt_forward(lens, Hq, Hk, D, dtype):
    q, k, v, _, cu = prompt_inputs(lens, Hq, Hk, D, dtype)
    out, lse = Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cu.cuda())
    assert E.evo_attn_device_status() == 0
    check_prompt(q, k, v, lens, out, lse, D ** -0.5, dtype)


def test_prompt_many_sequences():
    """More sequences than a warp reads at once, most of them short, some empty."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 9, 300)]
    lens[37], lens[250] = 200, 150
    q, k, v, do, cu = prompt_inputs(lens, 4, 2, 64, BF, seed=6)
    d = [x.cuda() for x in (q, k, v)]
    out, lse = Q.evo_prompt_fwd(*d, cu.cuda())
    check_prompt(q, k, v, lens, out, lse, 64 ** -0.5, BF)
    g = Q.evo_prompt_bwd(*d, cu.cuda(), out, lse, do.cuda())
    a = 0
    for n in lens:
        r = slice(a, a + n)
        a += n
        if n:
            S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x[r]) for x in g], 64 ** -0.5, BF)
    assert E.evo_attn_device_status() == 0


def test_prompt_rows_outside_and_scale():
    """Rows in front of the first and behind the last sequence are left alone; a scale."""
    lens = [70, 130]
    q, k, v, do, _ = prompt_inputs(lens, 4, 2, 64, BF, extra=33)
    cu = (S.offsets(lens) + 5).cuda()
    d = [x.cuda() for x in (q, k, v, do)]
    out, lse = torch.full_like(d[0], 7.0), torch.full((4, 233), 7.0, device="cuda")
    Q.evo_prompt_fwd(*d[:3], cu, out=out, lse=lse, scale=0.3)
    check_prompt(q, k, v, lens, out, lse, 0.3, BF, begin=5)
    grads = [torch.full_like(x, 7.0) for x in d[:3]]
    Q.evo_prompt_bwd(*d[:3], cu, out, lse, d[3], *grads, scale=0.3)
    for t in [out] + grads:
        assert torch.all(t[:5] == 7) and torch.all(t[205:] == 7)
    assert torch.all(lse[:, :5] == 7) and torch.all(lse[:, 205:] == 7)
    for a, n in ((5, 70), (75, 130)):
        r = slice(a, a + n)
        S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x[r]) for x in grads], 0.3, BF)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,Hq,Hk,D", [c for c in PROMPTS if c[1] * sum(c[0]) < 6000])
def test_prompt_backward(lens, Hq, Hk, D, dtype):
    q, k, v, do, cu = prompt_inputs(lens, Hq, Hk, D, dtype, seed=1)
    d = [x.cuda() for x in (q, k, v)]
    out, lse = Q.evo_prompt_fwd(*d, cu.cuda())
    g = Q.evo_prompt_bwd(*d, cu.cuda(), out, lse, do.cuda())
    assert E.evo_attn_device_status() == 0
    a = 0
    for n in lens:
        r = slice(a, a + n)
        a += n
        if n:
            S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x[r]) for x in g], D ** -0.5,
                              dtype, f"sequence of {n}")
    again = Q.evo_prompt_bwd(*d, cu.cuda(), out, lse, do.cuda())
    for x, y in zip(g, again):
        assert torch.equal(x, y)


def test_prompt_long_offsets_and_repeat():
    """Enough work that rows are shared out over every SM; a repeat gives the same bytes."""
    lens = [2500, 1, 1499]
    q, k, v, do, cu = prompt_inputs(lens, 4, 2, 128, BF, seed=2)
    d = [x.cuda() for x in (q, k, v)]
    cud = cu.cuda()
    out, lse = Q.evo_prompt_fwd(*d, cud)
    out2, lse2 = Q.evo_prompt_fwd(*d, cud)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    check_prompt(q, k, v, lens, out, lse, 128 ** -0.5, BF)
    g, g2 = (Q.evo_prompt_bwd(*d, cud, out, lse, do.cuda()) for _ in range(2))
    a = 0
    for n in lens:
        r = slice(a, a + n)
        a += n
        S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x[r]) for x in g], 128 ** -0.5, BF)
    for x, y in zip(g, g2):
        assert torch.equal(x, y)


def test_prompt_rising_scores():
    """Scores that rise along a sequence, in some rows of a warp only: the running maximum
    has to move, far, more than once, in rows next to rows where it stays."""
    lens, D = [900], 64
    q, k, v, do, cu = prompt_inputs(lens, 2, 1, D, BF, seed=3)
    q[::3] *= 4
    k *= (1 + torch.arange(900) / 150).view(-1, 1, 1).to(BF)
    d = [x.cuda() for x in (q, k, v)]
    out, lse = Q.evo_prompt_fwd(*d, cu.cuda())
    check_prompt(q, k, v, lens, out, lse, D ** -0.5, BF)


def test_unseen_values_do_not_spread():
    """NaN and infinities in one sequence, and in a sequence's later tokens, reach neither the
    other sequences nor the earlier tokens."""
    lens = [100, 77, 200]
    for dtype, D, Hq, Hk in ((BF, 128, 8, 2), (FP, 64, 2, 2), (BF, 128, 2, 2), (BF, 128, 1, 1)):
        q, k, v, do, cu = prompt_inputs(lens, Hq, Hk, D, dtype, seed=4)
        clean = [x.clone() for x in (q, k, v)]
        for x, val in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (v, float("-inf"))):
            x[100 + 33: 177: 7] = val
        k[177 + 150], v[177 + 60], v[177 + 131, :, 3] = float("nan"), float("inf"), float("nan")
        out, lse = Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cu.cuda())
        S.check_forward(*(S.f64(x[:100]) for x in clean), S.f64(out[:100]), S.f64(lse[:, :100]), D ** -0.5, dtype, "first")
        S.check_forward(*(S.f64(x[100:133]) for x in clean), S.f64(out[100:133]), S.f64(lse[:, 100:133]), D ** -0.5,
                        dtype, "in front of the NaN")
        S.check_forward(*(S.f64(x[177:237]) for x in clean), S.f64(out[177:237]), S.f64(lse[:, 177:237]), D ** -0.5,
                        dtype, "in front of the infinity")
        # rows that see them: where the definition gives an infinity or a NaN, so does the kernel
        tail = S.f64(out[237:327])
        assert np.all(np.isposinf(tail[:70].reshape(70, Hq, D))), "an infinite value that is seen"
        assert np.all(np.isnan(tail[71:, :, 3])) and np.all(np.isposinf(tail[71:, :, :3]))
        assert np.all(np.isnan(S.f64(out[327:])))  # a NaN key
        cl = [x.cuda() for x in clean]
        o2, l2 = Q.evo_prompt_fwd(*cl, cu.cuda())
        g0 = Q.evo_prompt_bwd(*cl, cu.cuda(), o2, l2, do.cuda())
        g1 = Q.evo_prompt_bwd(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), out, lse, do.cuda())
        for x, y in zip(g0, g1):  # the first sequence's gradients
            assert torch.equal(x[:100], y[:100])


def test_prompt_strided_projection():
    """q, k, v as the parts of one projection; out and the gradients into padded rows."""
    T, Hq, Hk, D = 211, 4, 2, 64
    rng = np.random.default_rng(7)
    qkv = S.normal(rng, T, Hq + 2 * Hk, D, dtype=BF).cuda()
    do = S.normal(rng, T, Hq, D, dtype=BF).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    cu = S.offsets([100, 111]).cuda()
    ref, ref_lse = Q.evo_prompt_fwd(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    pad = torch.full((T, 2 * Hq, D), 7.0, dtype=BF, device="cuda")
    out, lse = Q.evo_prompt_fwd(q, k, v, cu, out=pad[:, Hq:])
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and torch.all(pad[:, :Hq] == 7)
    g = Q.evo_prompt_bwd(q.contiguous(), k.contiguous(), v.contiguous(), cu, ref, ref_lse, do)
    dqkv = torch.full_like(qkv, 7.0)
    d2 = Q.evo_prompt_bwd(q, k, v, cu, out, lse, do, torch.full_like(pad, 7.0)[:, :Hq], dqkv[:, :Hk], dqkv[:, Hk:2 * Hk])
    for x, y in zip(g, d2):
        assert torch.equal(x, y)
    assert torch.all(dqkv[:, 2 * Hk:] == 7)


def test_bad_offsets_are_recorded():
    q, k, v, do, _ = prompt_inputs([64], 2, 1, 64, BF)
    d = [x.cuda() for x in (q, k, v)]
    for cu in ([0, 40, 30], [-4, 64], [0, 65], [0, 20, 2000000000]):
        out, lse = torch.full_like(d[0], 7.0), torch.full((2, 64), 7.0, device="cuda")
        mine = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.evo_prompt_fwd(*d, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out, lse=lse, status=mine)
        assert int(mine) == 13
        if cu[1] in (40, 20):  # the good sequence in front is as usual
            check_prompt(q, k, v, [cu[1]], out, lse, 64 ** -0.5, BF)
        assert torch.all(out[cu[1] if 0 < cu[1] < 64 and cu[0] == 0 else 0:] == 7)
        grads = [torch.full_like(x, 7.0) for x in d]
        Q.evo_prompt_bwd(*d, torch.tensor(cu, dtype=torch.int32, device="cuda"), out, lse, do.cuda(), *grads)
        assert E.evo_attn_device_status() == 13 and E.evo_attn_device_status() == 0


def test_nothing_to_do():
    z = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    kz = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = Q.evo_prompt_fwd(z, kz, kz, cu)
    assert out.shape == z.shape and lse.shape == (4, 0)
    q, k, v, do, _ = prompt_inputs([3], 4, 2, 64, BF)
    Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cu)  # three rows in no sequence
    assert E.evo_attn_device_status() == 0


def test_autograd_prompt():
    lens = [90, 0, 45]
    q, k, v, do, cu = prompt_inputs(lens, 4, 2, 64, BF, seed=9, extra=4)
    leaves = [x.cuda().requires_grad_(True) for x in (q, k, v)]
    out = prompt_attention(*leaves, cu.cuda())
    assert torch.all(out[135:] == 0)
    (out.float() * do.cuda().float()).sum().backward()
    for a, n in ((0, 90), (90, 45)):
        r = slice(a, a + n)
        S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x.grad[r]) for x in leaves],
                          64 ** -0.5, BF)
    for x in leaves:
        assert torch.all(x.grad[135:] == 0)
    # a broadcast (stride 0) gradient
    x = q.cuda().requires_grad_(True)
    prompt_attention(x, k.cuda(), v.cuda(), cu.cuda()).sum().backward()
    y = q.cuda().requires_grad_(True)
    prompt_attention(y, k.cuda(), v.cuda(), cu.cuda()).backward(torch.ones_like(q).cuda())
    assert torch.equal(x.grad, y.grad)


def test_gradient_against_differences():
    """Directional differences of the kernel's own forward (fp16, small step sizes cannot be
    taken in 16 bits: the step is along a direction that fp16 holds exactly)."""
    q, k, v, do, cu = prompt_inputs([48], 2, 1, 64, FP, seed=11)
    q, k, v = ((x * 64).round() / 64 for x in (q, k, v))
    cud, dod = cu.cuda(), do.cuda()
    out, lse = Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cud)
    grads = Q.evo_prompt_bwd(q.cuda(), k.cuda(), v.cuda(), cud, out, lse, dod)
    rng = np.random.default_rng(12)
    for i in range(3):
        step = torch.from_numpy(rng.integers(-1, 2, tuple((q, k, v)[i].shape)).astype(np.float32) / 64).to(FP)
        f = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * step
            o, _ = Q.evo_prompt_fwd(*(t.cuda() for t in x), cud)
            f.append(float((o.double().cpu() * do.double()).sum()))
        want = float((grads[i].double().cpu() * step.double()).sum())
        # two outputs, each rounded: |dO| |O| 2^-11 * 2 per element at most, random signs (x 8 of
        # the root of the sum of squares); third-order term of the step below 1/64: 2 %
        noise = 8 * float((do.double() * out.double().cpu() * 2.0 ** -10).square().sum().sqrt())
        assert abs((f[0] - f[1]) / 2 - want) <= noise + 0.02 * abs(want) + 0.05, (i, f, want)


# ------------------------------------------------------------------------------ paged cache
def paged_case(chunks, ctx, Hq, Hk, D, page, dtype, seed=0, fill=float("nan"), cols=None):
    rng = np.random.default_rng(seed)
    kp, vp, table = S.make_cache(rng, [max(c, 1) for c in ctx] if cols is None else [cols * page] * len(ctx), page, Hk,
                                 D, dtype, fill=fill)
    ks, vs = [S.normal(rng, n, Hk, D, dtype=dtype) for n in ctx], [S.normal(rng, n, Hk, D, dtype=dtype) for n in ctx]
    for b in range(len(ctx)):
        S.fill_cache(kp, vp, table, b, ks[b], vs[b])
    q = S.normal(rng, sum(chunks), Hq, D, dtype=dtype, sigma=1.5)
    return q, kp, vp, table, S.offsets(chunks), torch.tensor(ctx, dtype=torch.int32), ks, vs


def check_paged(c, chunks, ctx, out, lse, scale, dtype, w0=None, w=None, skip=()):
    q, _, _, _, cu, _, ks, vs = c
    for b, n in enumerate(chunks):
        if b in skip:
            continue
        r = slice(int(cu[b]), int(cu[b]) + n)
        if n:
            (_, _, wo, p), rp = S.check_forward(S.f64(q[r]), S.f64(ks[b]), S.f64(vs[b]), S.f64(out[r]), S.f64(lse[:, r]),
                                                scale, dtype, f"sequence {b}")
        if w is not None:
            L = ctx[b]
            before, after = S.f64(w0[b]), S.f64(w[b])
            assert np.array_equal(after[:, L:], before[:, L:])
            if n and L:
                bound = S.weight_bound(p, rp, q.shape[1] // ks[b].shape[1])
                S.assert_close(after[:, :L], before[:, :L] + wo, bound + 2.0 ** -23 * (before[:, :L] + wo), f"weights {b}")
            else:
                assert np.array_equal(after, before)


PAGED = [([1], [1], 1, 1, 64, 16), ([1, 1, 1], [37, 128, 300], 8, 2, 128, 16), ([1], [2000], 4, 1, 128, 64),
         ([3, 1, 0, 40], [3, 129, 50, 333], 6, 2, 64, 32), ([130, 257], [130, 700], 4, 2, 128, 128),
         ([5, 7], [2, 7], 4, 4, 64, 16), ([1, 2], [0, 1], 2, 1, 64, 16), ([64], [1000], 5, 1, 96, 256),
         ([1] * 40, [3 + 17 * i for i in range(40)], 4, 1, 64, 16), ([2, 1], [900, 65], 24, 2, 128, 32),
         ([300, 1], [1200, 1500], 8, 1, 72, 64), ([16, 9], [500, 9], 16, 2, 40, 384)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("chunks,ctx,Hq,Hk,D,page", PAGED)
def test_paged_forward(chunks, ctx, Hq, Hk, D, page, weights, dtype):
    """Every place of the cache that holds no token is NaN."""
    c = paged_case(chunks, ctx, Hq, Hk, D, page, dtype)
    q, kp, vp, table, cu, lens, _, _ = c
    w0 = w = None
    if weights:
        w0 = torch.rand(len(ctx), Hk, max(max(ctx), 1) + 3)
        w = w0.cuda()
    out, lse = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), cu.cuda(), lens.cuda(), table.cuda(), weights=w)
    assert E.evo_attn_device_status() == 0
    check_paged(c, chunks, ctx, out, lse, D ** -0.5, dtype, w0, w)


def test_paged_repeat_is_the_same_bytes():
    chunks, ctx = [1, 1, 70, 300], [3000, 777, 900, 2200]
    q, kp, vp, table, cu, lens, ks, vs = c = paged_case(chunks, ctx, 8, 2, 128, 64, BF)
    d = [x.cuda() for x in (q, kp, vp, cu, lens, table)]
    runs = []
    for _ in range(2):
        w = torch.zeros(4, 2, 3000, device="cuda")
        runs.append(Q.evo_paged_fwd(*d, weights=w) + (w,))
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    check_paged(c, chunks, ctx, *runs[0][:2], 128 ** -0.5, BF, torch.zeros(4, 2, 3000), runs[0][2])


def test_paged_unseen_values_do_not_spread():
    """NaN and infinities in the later tokens of a chunk."""
    for Hq, Hk, D, dtype in ((4, 1, 128, BF), (2, 2, 64, FP)):
        chunks, ctx = [90, 150], [400, 150]
        q, kp, vp, table, cu, lens, ks, vs = c = paged_case(chunks, ctx, Hq, Hk, D, 16, dtype)
        for b, at in ((0, 360), (1, 70)):
            j = torch.arange(at, ctx[b], 3)
            vp[table[b].long()[j // 16], j % 16] = float("nan")
            kp[table[b].long()[(j + 1).clamp(max=ctx[b] - 1) // 16], (j + 1).clamp(max=ctx[b] - 1) % 16] = float("inf")
        out, lse = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), cu.cuda(), lens.cuda(), table.cuda())
        S.check_forward(S.f64(q[:50]), S.f64(ks[0][:360]), S.f64(vs[0][:360]), S.f64(out[:50]), S.f64(lse[:, :50]),
                        D ** -0.5, dtype, "a")
        S.check_forward(S.f64(q[90:160]), S.f64(ks[1][:70]), S.f64(vs[1][:70]), S.f64(out[90:160]),
                        S.f64(lse[:, 90:160]), D ** -0.5, dtype, "b")
        assert torch.isnan(out[50:90]).all() and torch.isnan(out[160:]).all()


def test_paged_interleaved_pages():
    """Keys and values of a page next to each other in one buffer."""
    chunks, ctx = [2, 33], [100, 180]
    q, kp, vp, table, cu, lens, ks, vs = c = paged_case(chunks, ctx, 4, 2, 64, 32, BF)
    both = torch.stack([kp, vp], 1).cuda()
    d = [x.cuda() for x in (cu, lens, table)]
    out, lse = Q.evo_paged_fwd(q.cuda(), both[:, 0], both[:, 1], *d)
    check_paged(c, chunks, ctx, out, lse, 64 ** -0.5, BF)
    ref, _ = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), *d)
    assert torch.equal(ref, out)


def test_bad_pages_and_lengths_are_recorded():
    chunks, ctx = [1, 4, 2], [90, 70, 40]
    q, kp, vp, table, cu, lens, ks, vs = c = paged_case(chunks, ctx, 4, 2, 64, 16, BF)
    d = [x.cuda() for x in (q, kp, vp, cu)]
    for what in ("page", "negative page", "length", "negative length", "weights"):
        t2, l2, w = table.clone(), lens.clone(), None
        if what == "page":
            t2[1, 2] = kp.shape[0]
        elif what == "negative page":
            t2[1, 0] = -1
        elif what == "length":
            l2[1] = table.shape[1] * 16 + 1
        elif what == "negative length":
            l2[1] = -5
        else:
            l2[1] = 91
            w = torch.zeros(3, 2, 90, device="cuda")
        mine = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = Q.evo_paged_fwd(*d, l2.cuda(), t2.cuda(), weights=w, status=mine)
        assert int(mine) == 13, what
        check_paged(c, chunks, ctx, out, lse, 64 ** -0.5, BF, skip=(1,))
        k = S.normal(np.random.default_rng(1), 7, 2, 64, dtype=BF).cuda()
        kc, vc = kp.cuda(), vp.cuda()
        if what != "weights":
            mine.zero_()
            t2[1, 4] = t2[1, 4] if "length" in what else -1  # the page of the new tokens
            Q.evo_cache_append(k, k, d[3], l2.cuda(), kc, vc, t2.cuda(), status=mine)
            assert int(mine) == 13, what


@pytest.mark.parametrize("dtype", [BF, FP])
def test_append(dtype):
    chunks, ctx = [1, 20, 0, 5], [17, 40, 9, 3]  # the last has two tokens too many: not written
    rng = np.random.default_rng(0)
    kp, vp, table = S.make_cache(rng, ctx, 16, 2, 72, dtype, fill=3.0)
    qkv = S.normal(rng, 26, 4, 72, dtype=dtype)
    k, v = qkv[:, :2], qkv[:, 2:]
    kc, vc = kp.cuda(), vp.cuda()
    d = qkv.cuda()
    Q.evo_cache_append(d[:, :2], d[:, 2:], S.offsets(chunks).cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), kc, vc,
                       table.cuda())
    a = 0
    for b, (n, L) in enumerate(zip(chunks, ctx)):
        for i in range(n):
            j = L - n + i
            if j >= 0:
                kp[table[b, j // 16], j % 16] = k[a + i]
                vp[table[b, j // 16], j % 16] = v[a + i]
        a += n
    assert torch.equal(kc.cpu(), kp) and torch.equal(vc.cpu(), vp)
    assert E.evo_attn_device_status() == 0


# ------------------------------------------------------------------------------ eviction
def evict_case(ctx, Hk, D, page, dtype, seed=0, ties=True):
    rng = np.random.default_rng(seed)
    kp, vp, table = S.make_cache(rng, ctx, page, Hk, D, dtype, fill=5.0)
    ks, vs = [S.normal(rng, n, Hk, D, dtype=dtype) for n in ctx], [S.normal(rng, n, Hk, D, dtype=dtype) for n in ctx]
    for b in range(len(ctx)):
        S.fill_cache(kp, vp, table, b, ks[b], vs[b])
    w = rng.random((len(ctx), Hk, max(ctx) + 5)).astype(np.float32)
    if ties:
        w = np.where(w < 0.5, np.floor(w * 16) / 16, w ** 4 * 9).astype(np.float32)
    return kp, vp, table, torch.tensor(ctx, dtype=torch.int32), torch.from_numpy(w), ks, vs


def check_evict(case, ctx, budget, recent, after, kept):
    kp, vp, table, _, w, ks, vs = case
    kc, vc, lens, wc = after
    assert lens.tolist() == [min(n, budget) for n in ctx]
    page = kp.shape[1]
    want_k, want_v, want_w = kp.clone(), vp.clone(), w.clone()
    for b, n in enumerate(ctx):
        for h in range(kp.shape[2]):
            places = O.choose(w[b, h].double().numpy(), n, budget, recent)
            assert kept[b, h].tolist() == places + [-1] * (budget - len(places)), (b, h)
            if n <= budget:
                continue
            to = torch.arange(budget)
            want_k[table[b].long()[to // page], to % page, h] = ks[b][places, h]
            want_v[table[b].long()[to // page], to % page, h] = vs[b][places, h]
            want_w[b, h, :budget] = w[b, h, places]
            want_w[b, h, budget:n] = 0
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert np.array_equal(wc.numpy(), want_w.numpy(), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ctx,budget,recent,Hk,D,page", [
    ([100, 30, 64, 65], 64, 7, 2, 64, 16), ([1], 1, 0, 1, 8, 16), ([2, 1, 0], 1, 1, 1, 8, 16), ([5000], 1000, 100, 2, 128, 64),
    ([300, 301], 300, 300, 3, 96, 32), ([9000, 2500], 4500, 0, 1, 72, 128), ([1500], 1, 0, 4, 40, 256),
    ([4097, 4096, 4095], 4096, 17, 1, 64, 16), ([700], 699, 0, 2, 128, 384)])
def test_evict(ctx, budget, recent, Hk, D, page, dtype):
    case = evict_case(ctx, Hk, D, page, dtype)
    kp, vp, table, lens, w, _, _ = case
    d = [x.cuda() for x in (kp, vp, table, lens, w)]
    kept = Q.evo_cache_evict(*d, budget, recent)
    assert E.evo_attn_device_status() == 0
    check_evict(case, ctx, budget, recent, [d[0].cpu(), d[1].cpu(), d[3], d[4].cpu()], kept.cpu())


def test_evict_special_weights():
    """Equal weights, signed zeros, infinities and NaN: the order is the oracle's."""
    ctx = [400, 400, 400]
    case = evict_case(ctx, 1, 64, 16, BF)
    w = case[4]
    w[0] = 0.25
    w[1, :, ::2] = float("nan")
    w[1, :, 1::4] = float("-inf")
    w[2] = torch.randn(w[2].shape)
    w[2, :, ::3] = 0.0
    w[2, :, 1::3] = -0.0
    w[2, :, ::50] = float("inf")
    for budget, recent in ((150, 20), (290, 0)):
        d = [x.clone().cuda() for x in case[:2]] + [case[2].cuda(), case[3].cuda(), w.cuda()]
        kept = Q.evo_cache_evict(*d, budget, recent)
        check_evict(case, ctx, budget, recent, [d[0].cpu(), d[1].cpu(), d[3], d[4].cpu()], kept.cpu())


def test_evict_bad_entries_are_recorded():
    ctx = [100, 90]
    case = evict_case(ctx, 2, 64, 16, BF)
    for what in ("page", "length"):
        kp, vp, table, lens, w = (x.clone().cuda() for x in case[:5])
        if what == "page":
            table[1, 3] = 1 << 30
        else:
            lens[1] = 1 << 30
        kept = Q.evo_cache_evict(kp, vp, table, lens, w, 40, 3)
        assert E.evo_attn_device_status() == 13
        assert kept[0, 0].tolist() == O.choose(case[4][0, 0].double().numpy(), 100, 40, 3)
        if what == "length":
            assert int(lens[1]) == 1 << 30 and torch.all(kept[1] == -1) and torch.equal(w[1].cpu(), case[4][1])


# ------------------------------------------------------------------------------ together
def test_serving_run():
    """A prompt, its rows into the cache, a chunk and single tokens over it with the sums of
    their weights, an eviction, and more tokens over what is left: each step against the
    oracle on the rows that the cache then holds."""
    rng = np.random.default_rng(21)
    Hq, Hk, D, page, dtype, budget, recent = 8, 2, 128, 16, BF, 150, 20
    lens = [170, 60]
    kp, vp, table = S.make_cache(rng, [400, 400], page, Hk, D, dtype)
    kp, vp, td = kp.cuda(), vp.cuda(), table.cuda()
    weights = torch.zeros(2, Hk, 400, device="cuda")
    held_k, held_v = [[] for _ in lens], [[] for _ in lens]  # the oracle's cache, per sequence [L, Hkv, D]
    summed = [np.zeros((Hk, 0)) for _ in lens]
    size = torch.zeros(2, dtype=torch.int32, device="cuda")
    held_k = [np.zeros((0, Hk, D)) for _ in lens]
    held_v = [np.zeros((0, Hk, D)) for _ in lens]

    def step(new, prompt=False):
        T, cu = sum(new), S.offsets(new).cuda()
        q, k, v = (S.normal(rng, T, h, D, dtype=dtype) for h in (Hq, Hk, Hk))
        size.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
        Q.evo_cache_append(k.cuda(), v.cuda(), cu, size, kp, vp, td)
        out, lse = Q.evo_paged_fwd(q.cuda(), kp, vp, cu, size, td, weights=weights)
        if prompt:
            out2, lse2 = Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cu)
        a = 0
        for b, n in enumerate(new):
            r = slice(a, a + n)
            a += n
            held_k[b] = np.concatenate([held_k[b], S.f64(k[r])])
            held_v[b] = np.concatenate([held_v[b], S.f64(v[r])])
            (_, _, w, _), _ = S.check_forward(S.f64(q[r]), held_k[b], held_v[b], S.f64(out[r]), S.f64(lse[:, r]), D ** -0.5,
                                              dtype, f"step {new} sequence {b}")
            if prompt:
                S.check_forward(S.f64(q[r]), held_k[b], held_v[b], S.f64(out2[r]), S.f64(lse2[:, r]), D ** -0.5, dtype)
            summed[b] = np.concatenate([summed[b], np.zeros((Hk, n))], 1) + w
            got = S.f64(weights[b, :, :summed[b].shape[1]])
            assert np.allclose(got, summed[b], rtol=1e-4, atol=1e-6)

    def evict():
        # the choice is made on the kernel's own sums; the oracle follows it
        w = S.f64(weights)
        kept = Q.evo_cache_evict(kp, vp, td, size, weights, budget, recent).cpu()
        for b in range(2):
            L = held_k[b].shape[0]
            keep = [O.choose(w[b, h], L, budget, recent) for h in range(Hk)]
            for h in range(Hk):
                assert [x for x in kept[b, h].tolist() if x >= 0] == keep[h]
            held_k[b] = np.stack([held_k[b][keep[h], h] for h in range(Hk)], 1)
            held_v[b] = np.stack([held_v[b][keep[h], h] for h in range(Hk)], 1)
            summed[b] = np.stack([summed[b][h, keep[h]] for h in range(Hk)])
        assert size.tolist() == [x.shape[0] for x in held_k]

    step(lens, prompt=True)
    step([1, 30])
    evict()
    for _ in range(3):
        step([1, 1])
    step([40, 70])
    evict()
    step([1, 1])
    assert E.evo_attn_device_status() == 0


def test_streams_and_captured_graphs():
    """Calls on a side stream, two at once, and a captured step replayed on new inputs."""
    lens = [300, 41]
    q, k, v, do, cu = prompt_inputs(lens, 4, 2, 128, BF, seed=13)
    d = [x.cuda() for x in (q, k, v, do, cu)]
    ref = Q.evo_prompt_fwd(*d[:3], d[4])
    gref = Q.evo_prompt_bwd(*d[:3], d[4], *ref, d[3])
    chunks, ctx = [1, 9], [260, 777]
    c = paged_case(chunks, ctx, 4, 2, 128, 16, BF)
    pd = [x.cuda() for x in c[:6]]
    args = (pd[0], pd[1], pd[2], pd[4], pd[5], pd[3])
    pref = Q.evo_paged_fwd(*args)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        o = Q.evo_prompt_fwd(*d[:3], d[4], stream=s1)
        p = Q.evo_paged_fwd(*args, stream=s2)
        g = Q.evo_prompt_bwd(*d[:3], d[4], *o, d[3], stream=s1)
        got.append((o, p, g))
    torch.cuda.synchronize()
    for o, p, g in got:
        for x, y in zip(o + p + g, ref + pref + gref):
            assert torch.equal(x, y)
    # capture: forward, backward, chunk with weights
    w = torch.zeros(2, 2, 800, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o = Q.evo_prompt_fwd(*d[:3], d[4])
        g = Q.evo_prompt_bwd(*d[:3], d[4], *o, d[3])
        p = Q.evo_paged_fwd(*args, weights=w)
    for x in d[:3]:
        x.copy_(x.flip(2))  # new inputs: the same values, the features in reverse
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_prompt(d[0].cpu(), d[1].cpu(), d[2].cpu(), lens, o[0], o[1], 128 ** -0.5, BF)
    assert torch.equal(p[0], pref[0]) and torch.equal(p[1], pref[1])
    w1 = torch.zeros(2, 2, 800, device="cuda")
    Q.evo_paged_fwd(*args, weights=w1)
    assert torch.allclose(w, 2 * w1, rtol=1e-6, atol=0)
    r = slice(0, 300)
    S.check_gradients(*(S.f64(d[i][r]) for i in (0, 1, 2, 3)), [S.f64(x[r]) for x in g], 128 ** -0.5, BF)
    assert E.evo_attn_device_status() == 0


def test_binding_refusals_on_device():
    q, k, v, do, cu = (x.cuda() for x in prompt_inputs([40], 4, 2, 64, BF))
    for bad in (dict(k=k[:, :, :32]), dict(q=q[:, :3]), dict(v=v.half()), dict(cu=cu.long()), dict(k=k[:20]),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(cu=cu.cpu()), dict(cu=cu[:, None])):
        a = dict(q=q, k=k, v=v, cu=cu)
        a.update(bad)
        with pytest.raises(ValueError):
            Q.evo_prompt_fwd(a["q"], a["k"], a["v"], a["cu"])
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q, k, v, cu, scale=-1.0)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q, k, v, cu, lse=torch.zeros(40, 4, device="cuda"))
    with pytest.raises(E.EvoAttnError):
        Q.evo_prompt_fwd(q, k, v, cu, out=q)  # aliases an input
    with pytest.raises(E.EvoAttnError):
        Q.evo_prompt_fwd(q, k, v, cu, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert E.evo_attn_device_status() == 0


# ------------------------------------------------------------------------------ at the edges
def test_cache_offsets_past_32_bits():
    """Pages whose elements lie past 2^32: append, attention with weights, eviction."""
    Hk, D, page, pages, dtype = 8, 128, 64, 70000, BF
    kp = torch.empty(pages, page, Hk, D, dtype=dtype, device="cuda")
    vp = torch.empty_like(kp)
    assert kp.numel() > 2 ** 32
    rng = np.random.default_rng(31)
    table = torch.tensor([[69999, 65537, 69000], [66001, 68999, 69998]], dtype=torch.int32)
    lens, chunks = [150, 130], [150, 130]
    k, v = S.normal(rng, 280, Hk, D, dtype=dtype), S.normal(rng, 280, Hk, D, dtype=dtype)
    q = S.normal(rng, 280, 16, D, dtype=dtype)
    cu, size, td = S.offsets(chunks).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    Q.evo_cache_append(k.cuda(), v.cuda(), cu, size, kp, vp, td)
    w = torch.zeros(2, Hk, 192, device="cuda")
    out, lse = Q.evo_paged_fwd(q.cuda(), kp, vp, cu, size, td, weights=w)
    ref, ref_lse = Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cu)
    a = 0
    for b, n in enumerate(lens):
        r = slice(a, a + n)
        a += n
        (_, _, wo, p), rp = S.check_forward(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(out[r]), S.f64(lse[:, r]),
                                            D ** -0.5, dtype)
        S.assert_close(S.f64(w[b, :, :n]), wo, S.weight_bound(p, rp, 2) + 2.0 ** -23 * wo, "weights")
        kept = [O.choose(S.f64(w[b, h]), n, 100, 10) for h in range(Hk)]
        rows = [k[r][kept[h], h] for h in range(Hk)]
        if b == 0:
            want = rows
    Q.evo_cache_evict(kp, vp, td, size, w, 100, 10)
    got = kp[td[0].long()].view(-1, Hk, D)[:100]
    assert torch.equal(got.cpu(), torch.stack(want, 1))
    assert size.tolist() == [100, 100] and E.evo_attn_device_status() == 0


def test_rows_past_32_bits():
    """Token rows a long way apart."""
    T, Hq, Hk, D, stride = 300, 2, 1, 64, 1 << 24
    big = torch.empty(T * stride, dtype=BF, device="cuda")
    q = big.as_strided((T, Hq, D), (stride, D, 1))
    rng = np.random.default_rng(32)
    qh, k, v, do = (S.normal(rng, T, h, D, dtype=BF) for h in (Hq, Hk, Hk, Hq))
    q.copy_(qh)
    cu = S.offsets([T]).cuda()
    out = big[Hq * D:].as_strided((T, Hq, D), (stride, D, 1))
    kd, vd, dod = k.cuda(), v.cuda(), do.cuda()
    Q.evo_prompt_fwd(q, kd, vd, cu, out=out)
    o2, lse = Q.evo_prompt_fwd(qh.cuda(), kd, vd, cu)
    assert torch.equal(out, o2)
    dq = big[2 * Hq * D:].as_strided((T, Hq, D), (stride, D, 1))
    Q.evo_prompt_bwd(q, kd, vd, cu, out, lse, dod, dq)
    g = Q.evo_prompt_bwd(qh.cuda(), kd, vd, cu, o2, lse, dod)
    assert torch.equal(dq, g[0])


def test_shared_pages():
    """Two sequences that share the pages of a common beginning."""
    rng = np.random.default_rng(33)
    Hq, Hk, D, page = 4, 2, 64, 32
    kp, vp, table = S.make_cache(rng, [200, 200], page, Hk, D, BF)
    common = S.normal(rng, 96, 2 * Hk, D, dtype=BF)
    table[1, :3] = table[0, :3]
    ks, vs = [], []
    for b, n in enumerate((150, 170)):
        own = S.normal(rng, n - 96, 2 * Hk, D, dtype=BF)
        rows = torch.cat([common, own])
        ks.append(rows[:, :Hk].contiguous())
        vs.append(rows[:, Hk:].contiguous())
        S.fill_cache(kp, vp, table, b, ks[b], vs[b])
    q = S.normal(rng, 3, Hq, D, dtype=BF)
    cu, lens = S.offsets([1, 2]), torch.tensor([150, 170], dtype=torch.int32)
    w = torch.zeros(2, Hk, 200, device="cuda")
    out, lse = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), cu.cuda(), lens.cuda(), table.cuda(), weights=w)
    check_paged((q, kp, vp, table, cu, lens, ks, vs), [1, 2], [150, 170], out, lse, D ** -0.5, BF, torch.zeros(2, Hk, 200), w)


def test_many_empty_sequences():
    """Thousands of sequences, nearly all of them empty or done."""
    rng = np.random.default_rng(34)
    B, Hq, Hk, D, page = 5000, 2, 1, 64, 16
    chunks = np.zeros(B, dtype=np.int64)
    chunks[[0, 1234, 1235, 4999]] = [3, 1, 200, 2]
    ctx = rng.integers(0, 20, B)
    ctx[[0, 1234, 1235, 4999]] = [3, 60, 230, 17]
    kp, vp, table = S.make_cache(rng, [240], page, Hk, D, BF)
    pages = torch.from_numpy(rng.permutation(100).astype(np.int32))
    kp = torch.full((100, page, Hk, D), float("nan"), dtype=BF)
    vp = kp.clone()
    table = torch.zeros(B, 15, dtype=torch.int32)
    at, ks, vs = 0, {}, {}
    for b in (0, 1234, 1235, 4999):
        need = -(-int(ctx[b]) // page)
        table[b, :need] = pages[at:at + need]
        at += need
        ks[b], vs[b] = (S.normal(rng, int(ctx[b]), Hk, D, dtype=BF) for _ in range(2))
        S.fill_cache(kp, vp, table, b, ks[b], vs[b])
    q = S.normal(rng, int(chunks.sum()), Hq, D, dtype=BF)
    cu = S.offsets(chunks)
    w = torch.zeros(B, Hk, 240, device="cuda")
    out, lse = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), cu.cuda(), torch.from_numpy(ctx.astype(np.int32)).cuda(),
                               table.cuda(), weights=w)
    assert E.evo_attn_device_status() == 0
    for b in (0, 1234, 1235, 4999):
        r = slice(int(cu[b]), int(cu[b + 1]))
        (_, _, wo, p), rp = S.check_forward(S.f64(q[r]), S.f64(ks[b]), S.f64(vs[b]), S.f64(out[r]), S.f64(lse[:, r]),
                                            D ** -0.5, BF)
        S.assert_close(S.f64(w[b, :, :int(ctx[b])]), wo, S.weight_bound(p, rp, 2) + 2.0 ** -23 * wo, "weights")
    w[[0, 1234, 1235, 4999]] = 0
    assert torch.all(w == 0)


def test_a_wait_limit_and_a_status_word_of_the_callers():
    q, k, v, do, cu = (x.cuda() for x in prompt_inputs([200, 3], 4, 2, 64, BF))
    mine = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = Q.evo_prompt_fwd(q, k, v, cu, status=mine, wait_limit_ns=10 ** 9)
    Q.evo_prompt_bwd(q, k, v, cu, out, lse, do, status=mine, wait_limit_ns=10 ** 9)
    assert int(mine) == 0 and E.evo_attn_device_status() == 0
    check_prompt(q.cpu(), k.cpu(), v.cpu(), [200, 3], out, lse, 64 ** -0.5, BF)


def test_expanded_key_heads_gather_their_gradient():
    """Keys given as one head broadcast to two: the gradient is the sum over both."""
    q, k, v, do, cu = prompt_inputs([77], 4, 1, 64, BF, seed=40)
    cud = cu.cuda()
    one_k, one_v = k.cuda().requires_grad_(True), v.cuda().requires_grad_(True)
    out = prompt_attention(q.cuda(), one_k.expand(77, 2, 64), one_v.expand(77, 2, 64), cud)
    out.backward(do.cuda())
    g = Q.evo_prompt_bwd(q.cuda(), k.cuda(), v.cuda(), cud, *Q.evo_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cud), do.cuda())
    # two heads' gradients, rounded, then added and rounded: three roundings of at most their sizes
    for got, want in ((one_k.grad, g[1]), (one_v.grad, g[2])):
        size = float(want.abs().max())
        assert float((got.float() - want.float()).abs().max()) <= 6 * 2.0 ** -8 * size


def test_autograd_of_odd_gradients():
    """A gradient that starts off 16 bytes is copied; a second derivative is refused, not dropped."""
    q, k, v, do, cu = prompt_inputs([40, 9], 4, 2, 64, BF, seed=41)
    leaves = [x.cuda().requires_grad_(True) for x in (q, k, v)]
    buf = torch.empty(do.numel() + 1, dtype=BF, device="cuda")
    odd = buf[1:].view(do.shape)
    odd.copy_(do)
    assert odd.data_ptr() % 16
    grads = []
    for g in (do.cuda(), odd):
        out = prompt_attention(*leaves, cu.cuda())
        grads.append(torch.autograd.grad(out, leaves, g))
    for x, y in zip(*grads):
        assert torch.equal(x, y)
    out = prompt_attention(*leaves, cu.cuda())
    (dq,) = torch.autograd.grad(out, leaves[:1], do.cuda().requires_grad_(True), create_graph=True)
    with pytest.raises(RuntimeError):
        dq.sum().backward()


def test_offsets_that_share_rows():
    """Sequences with more rows than the call has, by offsets out of order: recorded, and nothing done."""
    q, k, v, do, _ = prompt_inputs([64], 2, 1, 64, BF, seed=42)
    d = [x.cuda() for x in (q, k, v)]
    for cu in ([0, 64, 0, 64], [0, 40, 10, 50], [0, 64] * 50 + [0, 60]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(d[0], 7.0), torch.full((2, 64), 7.0, device="cuda")
        mine = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.evo_prompt_fwd(*d, cud, out=out, lse=lse, status=mine)
        assert int(mine) == 13 and torch.all(out == 7) and torch.all(lse == 7)
        grads = [torch.full_like(x, 7.0) for x in d]
        Q.evo_prompt_bwd(*d, cud, out, torch.zeros_like(lse), do.cuda(), *grads)
        assert E.evo_attn_device_status() == 13 and all(bool(torch.all(x == 7)) for x in grads)
        # over a cache, the weights from the scores (many sequences) and formed again (few)
        B = len(cu) - 1
        pages = torch.zeros(16 * B, 16, 1, 64, dtype=BF, device="cuda")
        table = torch.arange(16 * B, dtype=torch.int32, device="cuda").view(B, 16)
        lens = torch.full((B,), 100, dtype=torch.int32, device="cuda")
        w = torch.full((B, 1, 256), 7.0, device="cuda")
        Q.evo_paged_fwd(d[0], pages, pages, cud, lens, table, out=out, lse=lse, weights=w)
        assert E.evo_attn_device_status() == 13
        assert torch.all(out == 7) and torch.all(lse == 7) and torch.all(w == 7)


@pytest.mark.parametrize("T,Hq,Hk,D,dtype", [(4099, 8, 8, 40, BF), (3300, 12, 4, 64, FP)])
def test_prompt_backward_of_much_work(T, Hq, Hk, D, dtype):
    """Enough work that every CTA does dK, dV and then dQ; two kv heads against the oracle."""
    q, k, v, do, cu = prompt_inputs([T], Hq, Hk, D, dtype, seed=43)
    d = [x.cuda() for x in (q, k, v, cu)]
    out, lse = Q.evo_prompt_fwd(*d)
    g = Q.evo_prompt_bwd(*d, out, lse, do.cuda())
    again = Q.evo_prompt_bwd(*d, out, lse, do.cuda())
    for x, y in zip(g, again):
        assert torch.equal(x, y)
    G = Hq // Hk
    for h in (0, Hk - 1):
        hq, hk = slice(h * G, (h + 1) * G), slice(h, h + 1)
        S.check_gradients(S.f64(q[:, hq]), S.f64(k[:, hk]), S.f64(v[:, hk]), S.f64(do[:, hq]),
                          [S.f64(g[0][:, hq]), S.f64(g[1][:, hk]), S.f64(g[2][:, hk])], D ** -0.5, dtype)
    assert E.evo_attn_device_status() == 0


def long_cache(L, page, D, dtype, seed):
    """A cache of L places that goes over the same four pages again and again: (k, v [4·page, D] fp64, k_pages,
    v_pages, table, how often each of the 4·page rows is there)."""
    rng = np.random.default_rng(seed)
    k, v = S.normal(rng, 4, page, 1, D, dtype=dtype), S.normal(rng, 4, page, 1, D, dtype=dtype)
    table = (torch.arange(-(-L // page), dtype=torch.int32) % 4)[None].contiguous()
    rows = 4 * page
    times = L // rows + (np.arange(rows) < L % rows)
    return S.f64(k).reshape(rows, D), S.f64(v).reshape(rows, D), k.cuda(), v.cuda(), table.cuda(), times


def check_long(q, k, v, times, L, out, lse, w, scale, dtype):
    """One token over long_cache's: every place of a row has the row's weight.  Bounds as in seq_util; l, O and
    the weights are sums of L/128 tiles, one rounding each, in whatever order."""
    G = q.shape[0]
    x = scale * (q @ k.T)
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    total = (e * times).sum(1)
    z, p = m[:, 0] + np.log(total), e / total[:, None]
    es, u = S.score_error(q[None], k[:, None], scale), S.U[dtype]
    adds = (L / 128 + 256) * 2.0 ** -24
    S.assert_close(S.f64(lse[:, 0]), z, es + 2.0 ** -19 * (1 + np.abs(z)) + adds, "lse")
    rp = 2 * es + 2.0 ** -18 * (1 + np.abs(z)) + 2 * adds
    S.assert_close(S.f64(out[0]), (p * times) @ v, (2 * u + rp[:, None]) * ((p * times) @ np.abs(v)) +
                   L * S.TINY[dtype] * np.max(np.abs(v)), "out")
    if w is not None:
        want, bound = p.sum(0), (p * (rp[:, None] + G * 2.0 ** -24)).sum(0)
        rows = k.shape[0]
        got = S.f64(w)
        for a in range(0, L, 1024 * rows):  # some million places at a time
            n = min(1024 * rows, L - a)
            idx = np.arange(n) % rows
            S.assert_close(got[a:a + n], want[idx], bound[idx], f"weights from {a}")
        assert np.all(got[L:] == 0)


def test_weights_of_a_wide_group_over_millions_of_keys():
    """(place of the key - place of the row) x heads of the group passes 2^31."""
    L, G, D, dtype = 23_000_000, 96, 8, BF
    k, v, kp, vp, table, times = long_cache(L, 1024, D, dtype, 51)
    q = S.normal(np.random.default_rng(52), 1, G, D, dtype=dtype)
    w = torch.zeros(1, 1, L + 5, device="cuda")
    out, lse = Q.evo_paged_fwd(q.cuda(), kp, vp, S.offsets([1]).cuda(), torch.tensor([L], dtype=torch.int32).cuda(), table,
                               weights=w)
    assert E.evo_attn_device_status() == 0
    check_long(S.f64(q[0]), k, v, times, L, out, lse, w[0, 0], D ** -0.5, dtype)


def test_evict_the_longest_sequence():
    """2^31 - 1025 places: the passes over them end past 2^31."""
    L, page, D, budget, recent = 2 ** 31 - 1025, 1024, 8, 600, 10
    cols = -(-L // page)
    gen = torch.Generator(device="cuda").manual_seed(61)
    kp = torch.empty(cols, page, 1, D, dtype=BF, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.randperm(cols, generator=gen, device="cuda").to(torch.int32)[None].contiguous()
    rng = np.random.default_rng(62)
    n, old = L - recent, budget - recent
    # the heaviest places: anywhere, the first, and the last ones of the passes
    some = sorted({0, 5000, n - 1, n - 2, n - 1024, n - 5000, n - 8192} | {int(x) for x in rng.integers(0, n, old)})
    drop = rng.permutation(range(1, len(some) - 7))[:len(some) - old]
    some = [x for i, x in enumerate(some) if i not in set(drop.tolist())]
    assert len(some) == old
    places = torch.tensor(some + list(range(n, L)), device="cuda")
    w = torch.zeros(1, 1, L + 3, device="cuda")
    w[0, 0, places[:old]] = torch.rand(old, generator=gen, device="cuda") + 0.5
    w[0, 0, n:L] = 0.25
    at = table[0].long()[places // page], places % page
    rows = torch.randn(2, budget, 1, D, generator=gen, device="cuda").to(BF)
    kp[at], vp[at] = rows[0], rows[1]
    want_w = w[0, 0, places].clone()
    size = torch.tensor([L], dtype=torch.int32, device="cuda")
    kept = Q.evo_cache_evict(kp, vp, table, size, w, budget, recent)
    assert E.evo_attn_device_status() == 0 and size.tolist() == [budget]
    assert torch.equal(kept[0, 0].long(), places)
    to = torch.arange(budget, device="cuda")
    for pages, want in ((kp, rows[0]), (vp, rows[1])):
        assert torch.equal(pages[table[0].long()[to // page], to % page], want)
    assert torch.equal(w[0, 0, :budget], want_w)
    assert int(torch.count_nonzero(w[0, 0, budget:])) == 0


def test_a_wait_that_runs_out():
    """The least limit, in calls whose first item takes a CTA some 65 000 sequences to find: recorded, in time, and
    the next calls are as ever.  (What a kernel that gave up has under way it still waits for, by a limit of its own.)"""
    B, T, Hq, Hk, D, page = 65535, 700, 4, 2, 64, 16
    q, k, v, do, _ = (x.cuda() if x is not None else x for x in prompt_inputs([T], Hq, Hk, D, BF, seed=71))
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[-1] = T
    cu = cu.cuda()
    cols = -(-T // page)
    kp, vp = (torch.zeros(3 * cols, page, Hk, D, dtype=BF, device="cuda") for _ in range(2))
    table = torch.zeros(B, cols, dtype=torch.int32, device="cuda")
    table[-1] = torch.arange(cols, device="cuda").flip(0)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = T
    Q.evo_cache_append(k, v, cu, lens, kp, vp, table)
    cu1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ref = Q.evo_prompt_fwd(q, k, v, cu1)
    gref = Q.evo_prompt_bwd(q, k, v, cu1, *ref, do)
    check_prompt(q.cpu(), k.cpu(), v.cpu(), [T], *ref, D ** -0.5, BF)

    def calls(limit, status):
        kw = dict(wait_limit_ns=limit, status=status)
        w = torch.zeros(B, Hk, T, device="cuda")
        o = Q.evo_prompt_fwd(q, k, v, cu, **kw)
        yield o
        yield Q.evo_prompt_bwd(q, k, v, cu, *(ref if limit else o), do, **kw)
        yield Q.evo_paged_fwd(q, kp, vp, cu, lens, table, weights=w, **kw)

    mine = torch.zeros(1, dtype=torch.int32, device="cuda")
    gave_up = []
    for _ in calls(1, mine):
        gave_up.append(int(mine))
        mine.zero_()
    # (a wait looks at its limit between some hundred tries: the forward's search may end within them)
    assert gave_up[1] == 8 and set(gave_up) <= {0, 8}, gave_up
    usual = list(calls(0, mine))
    assert int(mine) == 0 and E.evo_attn_device_status() == 0
    for b, (got, want) in enumerate(zip(usual, (ref, gref, ref))):
        for x, y in zip(got, want):
            # (another share of the work: other sums' order)
            assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -6, atol=2.0 ** -6), b


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_of_minus_infinity_give_no_weight(dtype):
    """A row whose every visible score is -inf gives 0, -inf and no weight, whether the weights are summed from the
    forward's scores (a token a sequence) or from scores formed again (many), beside rows as usual."""
    for chunks, ctx in (([1, 1, 1], [200, 131, 90]), ([40, 50, 30], [200, 131, 90])):
        q, kp, vp, table, cu, lens, ks, vs = c = paged_case(chunks, ctx, 4, 2, 64, 16, dtype, seed=81)
        r = slice(int(cu[1]), int(cu[2]))
        q[r, :, 0] = 1.0
        ks[1][:, :, 0] = float("-inf")
        S.fill_cache(kp, vp, table, 1, ks[1], vs[1])
        w0 = torch.rand(3, 2, 210)
        w = w0.cuda()
        out, lse = Q.evo_paged_fwd(q.cuda(), kp.cuda(), vp.cuda(), cu.cuda(), lens.cuda(), table.cuda(), weights=w)
        assert E.evo_attn_device_status() == 0
        assert torch.all(out[r] == 0) and torch.all(lse[:, r] == float("-inf"))
        assert torch.equal(w[1].cpu(), w0[1])
        check_paged(c, chunks, ctx, out, lse, 64 ** -0.5, dtype, w0, w, skip=(1,))


@pytest.mark.parametrize("L,G,D,page,room", [(40000, 8, 128, 16, True), (40000, 20, 64, 64, False),
                                             (131071, 4, 128, 128, True), (131071, 1, 72, 16, False)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_one_long_context_over_every_sm(L, G, D, page, room, dtype):
    """One token, one kv head, one sequence: an item cut into a piece for every CTA, more than the join looks at in
    one go; the weights from the forward's scores (a cache with room) and formed again (a small one)."""
    k, v, kp, vp, table, times = long_cache(L, page, D, dtype, 91)
    if room:  # pages in no table
        kp, vp = (torch.cat([x, x.new_full((-(-L // page), page, 1, D), float("nan"))]) for x in (kp, vp))
    q = S.normal(np.random.default_rng(92), 1, G, D, dtype=dtype, sigma=1.5)
    d = (q.cuda(), kp, vp, S.offsets([1]).cuda(), torch.tensor([L], dtype=torch.int32).cuda(), table)
    w = torch.zeros(1, 1, L + 5, device="cuda")
    need = [Q.evo_paged_fwd_workspace_bytes(1, 1, G, 1, D, kp.shape[0], page, table.shape[1], n) for n in (0, L + 5)]
    assert (need[1] > need[0]) == room
    out, lse = Q.evo_paged_fwd(*d, weights=w)
    out2, lse2 = Q.evo_paged_fwd(*d)
    assert E.evo_attn_device_status() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    check_long(S.f64(q[0]), k, v, times, L, out, lse, w[0, 0], D ** -0.5, dtype)


def test_evict_more_pages_than_the_moves_hold():
    """4375 pages of one sequence, places read and written beyond the first 4096 of them."""
    ctx, budget, recent = [70000], 66000, 100
    case = evict_case(ctx, 1, 8, 16, BF, seed=93)
    d = [x.cuda() for x in case[:5]]
    kept = Q.evo_cache_evict(*d, budget, recent)
    assert E.evo_attn_device_status() == 0
    check_evict(case, ctx, budget, recent, [d[0].cpu(), d[1].cpu(), d[3], d[4].cpu()], kept.cpu())


def test_rejected_sequences_get_no_gradient():
    """Rows of a sequence with a bad offset keep what the gradients held, the good one in front is as usual."""
    q, k, v, do, _ = prompt_inputs([64], 2, 1, 64, BF)
    d = [x.cuda() for x in (q, k, v, do)]
    for cu, good in (([0, 40, 30], 40), ([-4, 64], 0), ([0, 65], 0), ([0, 20, 2000000000], 20)):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(d[0], 7.0), torch.full((2, 64), 7.0, device="cuda")
        mine = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.evo_prompt_fwd(*d[:3], cud, out=out, lse=lse, status=mine)
        grads = [torch.full_like(x, 7.0) for x in d[:3]]
        Q.evo_prompt_bwd(*d[:3], cud, out, lse, d[3], *grads, status=mine)
        assert int(mine) == 13
        for t in [out] + grads:
            assert torch.all(t[good:] == 7), cu
        if good:
            r = slice(0, good)
            S.check_gradients(S.f64(q[r]), S.f64(k[r]), S.f64(v[r]), S.f64(do[r]), [S.f64(x[r]) for x in grads], 64 ** -0.5, BF)
    assert E.evo_attn_device_status() == 0
