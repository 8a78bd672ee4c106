"""Host-side refusals of the causal-sequence entry points: the C ABI's validation, which
answers before anything reaches a GPU, and the binding's (CPU only)."""
import ctypes

import pytest
import torch

from memory_efficient_biased_gb300 import evo_seq as Q
from memory_efficient_biased_gb300.autograd import _packed_rows

A = 1 << 32  # fake, well-aligned device addresses far apart: validation never dereferences them
REACH = (0, 6, 7)  # valid arguments reach the device check


@pytest.fixture(scope="module")
def lib():
    from memory_efficient_biased_gb300 import build
    build.build()
    return Q.load()


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def shape(T=64, B=2, Hq=8, Hk=2, D=64):
    return Q.SeqShape(T, B, Hq, Hk, D)


def cache(P=10, page=16, cols=4, ks=0, vs=0):
    return Q.CacheShape(P, page, cols, ks, vs)


def opts(**kw):
    o = Q.SeqOptions()
    o.size = ctypes.sizeof(Q.SeqOptions)
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def ref(x):
    return None if x is None else ctypes.byref(x)


def fwd(lib, s=None, dt=1, strides=None, o=None, ws_bytes=None, **p):
    s = s or shape()
    a = dict(q=A, k=2 * A, v=3 * A, cu=4 * A, out=5 * A, lse=6 * A, ws=7 * A)
    a.update(p)
    need = lib.evo_prompt_fwd_workspace_bytes(s) if ws_bytes is None else ws_bytes
    return lib.evo_prompt_fwd(*(vp(a[n]) for n in ("q", "k", "v", "cu", "out", "lse", "ws")), need, s, dt, ref(strides),
                              o, None)


def bwd(lib, s=None, dt=1, strides=None, o=None, ws_bytes=None, **p):
    s = s or shape()
    a = dict(q=A, k=2 * A, v=3 * A, cu=4 * A, out=5 * A, lse=6 * A, do=8 * A, dq=9 * A, dk=10 * A, dv=11 * A, ws=7 * A)
    a.update(p)
    need = lib.evo_prompt_bwd_workspace_bytes(s) if ws_bytes is None else ws_bytes
    return lib.evo_prompt_bwd(*(vp(a[n]) for n in ("q", "k", "v", "cu", "out", "lse", "do", "dq", "dk", "dv", "ws")),
                              need, s, dt, ref(strides), o, None)


def append(lib, s=None, c=None, dt=1, strides=None, o=None, **p):
    a = dict(k=2 * A, v=3 * A, cu=4 * A, lens=12 * A, table=13 * A, kp=14 * A, vpg=15 * A)
    a.update(p)
    return lib.evo_cache_append(*(vp(a[n]) for n in ("k", "v", "cu", "lens", "table", "kp", "vpg")), s or shape(),
                                c or cache(), dt, ref(strides), o, None)


def paged(lib, s=None, c=None, dt=1, strides=None, o=None, ws_bytes=None, w=None, wlen=0, **p):
    s, c = s or shape(), c or cache()
    a = dict(q=A, kp=14 * A, vpg=15 * A, cu=4 * A, lens=12 * A, table=13 * A, out=5 * A, lse=6 * A, ws=7 * A)
    a.update(p)
    need = lib.evo_paged_fwd_workspace_bytes(s, c, wlen if w else 0) if ws_bytes is None else ws_bytes
    return lib.evo_paged_fwd(*(vp(a[n]) for n in ("q", "kp", "vpg", "cu", "lens", "table", "out", "lse")), vp(w), wlen,
                             vp(a["ws"]), need, s, c, dt, ref(strides), o, None)


def evict(lib, s=None, c=None, dt=1, o=None, wlen=64, budget=32, recent=4, **p):
    a = dict(kp=14 * A, vpg=15 * A, table=13 * A, lens=12 * A, w=16 * A, kept=17 * A)
    a.update(p)
    return lib.evo_cache_evict(*(vp(a[n]) for n in ("kp", "vpg", "table", "lens", "w")), wlen, vp(a["kept"]), budget,
                               recent, s or shape(), c or cache(), dt, o, None)


@pytest.mark.parametrize("call", [fwd, bwd, paged])
def test_attention_refusals(lib, call):
    assert call(lib) in REACH
    assert call(lib, dt=2) == 3
    for bad in (shape(D=12), shape(D=136), shape(D=0), shape(Hq=7), shape(Hk=0), shape(Hq=0), shape(T=-1), shape(B=-1),
                shape(Hq=258, Hk=2), shape(B=70000), shape(T=1 << 31)):
        assert call(lib, s=bad, ws_bytes=1 << 30) == 2, list(getattr(bad, n) for n, _ in bad._fields_)
    # nothing to do: no pointer is needed
    assert call(lib, s=shape(T=0), q=None, out=None) == 0
    assert call(lib, s=shape(B=0), q=None, out=None) == 0
    for name in ("q", "cu", "out", "lse", "ws"):
        assert call(lib, **{name: None}) == 1, name
    for name, off in (("q", 8), ("out", 2), ("cu", 2), ("lse", 2), ("ws", 128)):
        base = dict(q=A, out=5 * A, cu=4 * A, lse=6 * A, ws=7 * A)[name]
        assert call(lib, **{name: base + off}) == 4, name
    assert call(lib, ws_bytes=8) == 5
    assert call(lib, o=opts(flags=1)) == 10
    assert call(lib, o=opts(reserved=1)) == 10
    assert call(lib, o=opts(size=8)) == 10
    for scale in (-1.0, float("inf"), float("nan")):
        assert call(lib, o=opts(scale=scale)) == 10
    assert call(lib, o=opts(scale=0.25, wait_limit_ns=10)) in REACH
    assert call(lib, o=opts(status=2)) == 4
    # strides: multiples of 8, rows do not overlap
    for bad in (64, 516, -512, 1 << 36):
        assert call(lib, strides=Q.SeqStrides(q=bad)) == 12, bad
    assert call(lib, strides=Q.SeqStrides(q=768)) in REACH


def test_aliasing(lib):
    assert fwd(lib, out=A) == 9
    assert fwd(lib, lse=2 * A) == 9
    assert fwd(lib, lse=5 * A + 64) == 9
    assert fwd(lib, ws=3 * A) == 9
    assert fwd(lib, q=A, k=A + 1024, v=A + 1280, strides=Q.SeqStrides(q=768, k=768, v=768)) in REACH  # one projection
    for name in ("dq", "dk", "dv"):
        assert bwd(lib, **{name: 8 * A}) == 9
        assert bwd(lib, **{name: 5 * A}) == 9
    assert bwd(lib, dk=9 * A) == 9
    one = Q.SeqStrides(dq=768, dk=768, dv=768)  # the gradients as the parts of one projection's
    assert bwd(lib, strides=one, dq=9 * A, dk=9 * A + 1024, dv=9 * A + 1280) in REACH
    assert bwd(lib, strides=one, dq=9 * A, dk=9 * A + 1024, dv=9 * A + 1264) == 9
    assert bwd(lib, strides=one, dq=9 * A, dk=9 * A + 1280, dv=9 * A + 1536 + 1024 - 16) == 9
    assert paged(lib, out=14 * A) == 9
    assert paged(lib, w=6 * A, wlen=64) == 9
    assert append(lib, kp=2 * A) == 9
    assert append(lib, kp=15 * A) == 9
    one = 16 * 2 * 64
    inter = cache(ks=2 * one, vs=2 * one)  # keys and values interleaved page by page
    assert append(lib, c=inter, kp=14 * A, vpg=14 * A + one * 2) in REACH
    assert append(lib, c=inter, kp=14 * A, vpg=14 * A + one * 2 - 16) == 9
    assert append(lib, c=inter, kp=14 * A + one * 2, vpg=14 * A) in REACH
    assert evict(lib, c=inter, kp=14 * A, vpg=14 * A + one * 2) in REACH
    assert evict(lib, kept=14 * A) == 9
    assert evict(lib, kept=16 * A) == 9
    assert evict(lib, lens=13 * A) == 9


def test_cache_refusals(lib):
    for call in (append, paged, evict):
        assert call(lib) in REACH
        for bad in (cache(page=8), cache(page=48), cache(page=100), cache(page=2048), cache(P=0), cache(cols=0)):
            kw = {"ws_bytes": 1 << 30} if call is paged else {}
            assert call(lib, c=bad, **kw) == 2
        for stride in (16 * 2 * 64 - 8, 16 * 2 * 64 + 4, 1 << 36):
            kw = {"ws_bytes": 1 << 30} if call is paged else {}
            assert call(lib, c=cache(ks=stride), **kw) == 12, stride
        for name in ("kp", "vpg", "table", "lens"):
            assert call(lib, **{name: None}) == 1, name
        assert call(lib, kp=14 * A + 8) == 4
        assert call(lib, table=13 * A + 2) == 4
        assert call(lib, dt=5) == 3
    assert append(lib, s=shape(T=0), k=None) == 0
    assert paged(lib, w=16 * A, wlen=0) == 2
    assert paged(lib, w=16 * A + 2, wlen=64) == 4
    assert paged(lib, w=16 * A, wlen=64) in REACH


def test_evict_refusals(lib):
    assert evict(lib, s=shape(B=0), kp=None) == 0
    for kw in (dict(budget=0), dict(budget=-3), dict(recent=-1), dict(recent=33)):
        assert evict(lib, **kw) == 10, kw
    assert evict(lib, recent=32) in REACH
    assert evict(lib, recent=0) in REACH
    assert evict(lib, wlen=0) == 2
    assert evict(lib, kept=None) == 1
    assert evict(lib, kept=17 * A + 2) == 4
    assert evict(lib, w=None) == 1


def test_workspace_bytes(lib):
    assert lib.evo_prompt_fwd_workspace_bytes(shape()) % 256 == 0
    assert lib.evo_prompt_fwd_workspace_bytes(shape(D=12)) == 0
    assert lib.evo_prompt_bwd_workspace_bytes(shape(Hq=3)) == 0
    assert lib.evo_prompt_bwd_workspace_bytes(shape()) >= 64 * 8 * 4  # delta
    assert lib.evo_paged_fwd_workspace_bytes(shape(), cache(page=24), 0) == 0
    assert lib.evo_paged_fwd_workspace_bytes(shape(), cache(), -1) == 0
    need = lambda sh, c, w: lib.evo_paged_fwd_workspace_bytes(sh, c, w)
    assert need(shape(), cache(), 0) > 0
    # single tokens: room for the scores ([tokens][q_heads][length, in whole tiles] fp32) with weights ...
    one, c = shape(T=2), cache(P=40, cols=16)
    assert need(one, c, 200) == need(one, c, 0) + 2 * 8 * 256 * 4
    # ... unless they would be large beside the cache, or there are many rows a key
    small, many = cache(P=2, cols=16), shape(T=16)
    assert need(one, small, 256) == need(one, small, 0)
    assert need(many, c, 256) == need(many, c, 0)
    # little work needs few CTAs' worth of partial results
    assert need(shape(T=1, B=1), cache(), 0) < need(shape(T=4096, B=8), cache(P=4096, cols=1024), 0)
    assert lib.evo_prompt_fwd_workspace_bytes(shape(T=8)) < lib.evo_prompt_fwd_workspace_bytes(shape(T=8192))


def test_binding_refuses_host_tensors_and_shapes():
    """ValueError before anything reaches the library (no GPU here: every tensor is a host one)."""
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q, k, k, cu)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q[0], k, k, cu)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q.float(), k, k, cu)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q[:, :3], k, k, cu)
    with pytest.raises(ValueError):
        Q.evo_prompt_fwd(q, k, k, [0, 4])
    pages = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    lens, table = torch.tensor([4], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        Q.evo_paged_fwd(q, pages, pages, cu, lens, table)
    with pytest.raises(ValueError):
        Q.evo_cache_append(k, k, cu, lens, pages, pages, table)
    with pytest.raises(ValueError):
        Q.evo_cache_evict(pages, pages, table, lens, torch.zeros(1, 2, 32), 8)


def test_binding_page_strides():
    """Pages that overlap (one page expanded to several) are refused: their stride of 0 means packed below."""
    table, dt = torch.zeros(1, 2, dtype=torch.int32), torch.bfloat16
    one, many = torch.zeros(1, 16, 2, 64, dtype=dt), torch.zeros(4, 16, 2, 64, dtype=dt)
    for bad in (one.expand(4, 16, 2, 64), many.as_strided((4, 16, 2, 64), (1024, 128, 64, 1)),
                many[:, :, :1].expand(4, 16, 2, 64)):
        for pair in ((bad, many), (many, bad)):
            with pytest.raises(ValueError):
                Q._cache(*pair, table, 1, dt, -1)
    both = torch.zeros(4, 2, 16, 2, 64, dtype=dt)
    c = Q._cache(both[:, 0], both[:, 1], table, 1, dt, -1)
    assert (c.num_pages, c.page_size, c.pages_per_seq, c.k_page_stride, c.v_page_stride) == (4, 16, 2, 4096, 4096)


def test_binding_options():
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-60, 1e60):
        with pytest.raises(ValueError):
            Q._options(scale, 0, None, -1)
    for wait in (-1, 1 << 64):
        with pytest.raises(ValueError):
            Q._options(None, wait, None, -1)
    assert Q._options(None, 0, None, -1) is None
    o = Q._options(0.5, 7, None, -1)._obj
    assert (o.scale, o.wait_limit_ns, o.status) == (0.5, 7, None)


def test_packed_rows():
    """What the library cannot read in place is copied: a start off 16 bytes too, although contiguous."""
    for dt in (torch.bfloat16, torch.float16):
        buf = torch.randn(1 + 5 * 2 * 64).to(dt)
        odd = buf[1:].view(5, 2, 64)
        fused = torch.randn(5, 6, 64).to(dt)
        for t in (odd, fused.transpose(0, 1), fused[:1, :1].expand(5, 2, 64), torch.randn(5, 2, 64).to(dt)[::2, :, :60]):
            p = _packed_rows(t)
            assert p.data_ptr() % 16 == 0 and p.is_contiguous() and torch.equal(p, t)
        for t in (fused, fused[:, 2:4], fused[::2]):
            assert _packed_rows(t) is t


@pytest.mark.parametrize("call", [fwd, bwd, paged])
def test_scale_times_log2e_is_a_number(lib, call):
    """The kernels work with scale · log2 e in float32: a scale that is a number only without it is refused."""
    for scale in (2.36e38, 3.0e38, 3.4028234e38):
        assert call(lib, o=opts(scale=scale)) == 10, scale
        with pytest.raises(ValueError):
            Q._options(scale, 0, None, -1)
    for scale in (2.357e38, 1e-40):
        assert call(lib, o=opts(scale=scale)) in REACH, scale
        assert Q._options(scale, 0, None, -1)._obj.scale == ctypes.c_float(scale).value
