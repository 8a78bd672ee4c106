"""Host-side refusals of rotary positions and of the 8-bit cache: the C ABI's validation, which
answers before anything reaches a GPU, and the binding's (CPU only)."""
import ctypes

import pytest
import torch

from memory_efficient_biased_gb300 import evo_seq as Q
from tests.test_seq_host import A, REACH, opts, ref, shape, vp


@pytest.fixture(scope="module")
def lib():
    from memory_efficient_biased_gb300 import build
    build.build()
    return Q.load()


def rotary(lib, s=None, r=None, dt=1, strides=None, null=False, **p):
    a = dict(q=A, k=2 * A, pos=3 * A, freq=4 * A, qo=5 * A, ko=6 * A)
    a.update(p)
    r = r or Q.Rotary(64, 0, 1.0, 0, 0)
    return lib.evo_rotary(*(vp(a[n]) for n in ("q", "k", "pos", "freq", "qo", "ko")), s or shape(),
                          None if null else ctypes.byref(r), dt, ref(strides), None)


def cache(P=10, page=16, cols=4, block=16, ks=0, vs=0):
    return Q.Cache8Shape(P, page, cols, block, ks, vs)


def append(lib, s=None, c=None, dt=1, strides=None, o=None, **p):
    a = dict(k=2 * A, v=3 * A, cu=4 * A, lens=12 * A, table=13 * A, kp=14 * A, vpg=15 * A, ks=16 * A, vs=17 * A)
    a.update(p)
    return lib.evo_cache8_append(*(vp(a[n]) for n in ("k", "v", "cu", "lens", "table", "kp", "vpg", "ks", "vs")),
                                 s or shape(), c or cache(), dt, ref(strides), o, None)


def read(lib, s=None, c=None, dt=1, strides=None, o=None, **p):
    a = dict(k=2 * A, v=3 * A, cu=4 * A, lens=12 * A, table=13 * A, kp=14 * A, vpg=15 * A, ks=16 * A, vs=17 * A)
    a.update(p)
    return lib.evo_cache8_read(*(vp(a[n]) for n in ("kp", "vpg", "ks", "vs", "cu", "lens", "table", "k", "v")),
                               s or shape(), c or cache(), dt, ref(strides), o, None)


def paged(lib, s=None, c=None, dt=1, strides=None, o=None, ws_bytes=None, **p):
    s, c = s or shape(), c or cache()
    a = dict(q=A, kp=14 * A, vpg=15 * A, ks=16 * A, vs=17 * A, cu=4 * A, lens=12 * A, table=13 * A, out=5 * A, lse=6 * A,
             ws=7 * A)
    a.update(p)
    need = lib.evo_paged8_fwd_workspace_bytes(s, c) if ws_bytes is None else ws_bytes
    return lib.evo_paged8_fwd(*(vp(a[n]) for n in ("q", "kp", "vpg", "ks", "vs", "cu", "lens", "table", "out", "lse", "ws")),
                              need, s, c, dt, ref(strides), o, None)


def test_rotary_refusals(lib):
    assert rotary(lib) in REACH
    assert rotary(lib, k=None, ko=None) in REACH
    assert rotary(lib, null=True) == 1
    for name in ("q", "qo", "pos", "freq"):
        assert rotary(lib, **{name: None}) == 1, name
    assert rotary(lib, k=None) == 10 and rotary(lib, ko=None) == 10
    assert rotary(lib, r=Q.Rotary(64, 4, 1.0, 0, 0)) == 10
    for f in (float("inf"), float("nan")):
        assert rotary(lib, r=Q.Rotary(64, 0, f, 0, 0)) == 10
    assert rotary(lib, r=Q.Rotary(64, 3, 0.0, 0, 0)) in REACH
    assert rotary(lib, dt=2) == 3
    for dim in (0, 3, 66, -2):
        assert rotary(lib, r=Q.Rotary(dim, 0, 1.0, 0, 0)) == 2, dim
    for bad in (shape(D=12), shape(D=136), shape(D=0), shape(Hq=0), shape(Hq=65536), shape(T=-1), shape(T=1 << 31),
                shape(Hk=-1), shape(Hk=16385)):
        assert rotary(lib, s=bad) == 2
    assert rotary(lib, s=shape(Hq=7, Hk=3)) in REACH  # no groups here
    assert rotary(lib, s=shape(T=0), q=None, qo=None) == 0
    for name, base, off in (("q", A, 8), ("k", 2 * A, 2), ("qo", 5 * A, 8), ("ko", 6 * A, 8), ("pos", 3 * A, 2), ("freq", 4 * A, 4)):
        assert rotary(lib, **{name: base + off}) == 4, name
    for bad in (64, 516, -512, 1 << 36):
        assert rotary(lib, strides=Q.SeqStrides(q=bad)) == 12
        assert rotary(lib, r=Q.Rotary(64, 0, 1.0, bad, 0)) == 12
    assert rotary(lib, strides=Q.SeqStrides(k=64)) == 12
    assert rotary(lib, r=Q.Rotary(64, 0, 1.0, 0, 64)) == 12
    # in place, as it is; otherwise nothing overlaps
    assert rotary(lib, qo=A, ko=2 * A) in REACH
    one = Q.SeqStrides(q=768, k=768)
    part = Q.Rotary(64, 0, 1.0, 768, 768)
    assert rotary(lib, strides=one, r=part, q=A, k=A + 1024, qo=A, ko=A + 1024) in REACH
    assert rotary(lib, strides=one, r=part, q=A, k=A + 1024, qo=A, ko=A + 1008) == 9
    assert rotary(lib, strides=one, q=A, k=A + 1024, qo=A) == 9  # another stride
    assert rotary(lib, qo=A + 64) == 9
    assert rotary(lib, qo=2 * A) == 9
    assert rotary(lib, qo=5 * A, ko=5 * A) == 9
    assert rotary(lib, qo=3 * A) == 9 and rotary(lib, ko=4 * A) == 9


@pytest.mark.parametrize("call", [append, read, paged])
def test_cache8_refusals(lib, call):
    assert call(lib) in REACH
    assert call(lib, dt=2) == 3
    for bad in (shape(D=8), shape(D=72), shape(D=144), shape(D=0), shape(Hk=0), shape(T=-1), shape(B=-1), shape(B=70000),
                shape(T=1 << 31)):
        assert call(lib, s=bad, **({"ws_bytes": 1 << 30} if call is paged else {})) == 2
    for bad in (cache(page=24), cache(page=8), cache(page=2048), cache(block=8), cache(block=32), cache(page=64, block=48),
                cache(page=256, block=256), cache(block=0), cache(P=0), cache(cols=0), cache(page=384, block=256)):
        assert call(lib, c=bad, **({"ws_bytes": 1 << 30} if call is paged else {})) == 2
    assert call(lib, c=cache(page=384, block=128)) in REACH
    for bad in (16, 16 * 2 * 64 + 8, 1 << 36, -4096):
        assert call(lib, c=cache(ks=bad)) == 12
        assert call(lib, c=cache(vs=bad)) == 12
    empty = dict(q=None, out=None) if call is paged else dict(k=None, v=None)
    assert call(lib, s=shape(T=0), **empty) == 0
    assert call(lib, s=shape(B=0), **empty) == 0
    at = dict(kp=14 * A, vpg=15 * A, ks=16 * A, vs=17 * A, cu=4 * A, lens=12 * A, table=13 * A)
    at.update(dict(q=A, out=5 * A, lse=6 * A, ws=7 * A) if call is paged else dict(k=2 * A, v=3 * A))
    for name, base in at.items():
        assert call(lib, **{name: None}) == 1, name
        assert call(lib, **{name: base + 2}) == 4, name
    assert call(lib, kp=14 * A + 8) == 4
    assert call(lib, o=opts(flags=1)) == 10
    assert call(lib, o=opts(size=8)) == 10
    assert call(lib, o=opts(scale=-1.0)) == 10
    assert call(lib, o=opts(status=2)) == 4
    if call is paged:
        assert call(lib, ws_bytes=8) == 5
        assert call(lib, ws=7 * A + 128) == 4
        one = shape(T=2, B=2)  # single tokens over at most 64 places: no workspace
        assert lib.evo_paged8_fwd_workspace_bytes(one, cache()) == 0
        assert call(lib, s=one, ws=None) in REACH
        assert call(lib, s=one, c=cache(cols=100), ws=None) == 1
        assert call(lib, s=shape(Hq=7), ws_bytes=1 << 30) == 2
        assert call(lib, s=shape(Hq=258), ws_bytes=1 << 30) == 2
        assert call(lib, strides=Q.SeqStrides(q=516)) == 12


def test_cache8_aliasing(lib):
    one = 16 * 2 * 64  # a page, in bytes
    inter = cache(ks=2 * one, vs=2 * one)
    for call in (append, read, paged):
        assert call(lib, c=inter, kp=14 * A, vpg=14 * A + one) in REACH
    assert append(lib, c=inter, kp=14 * A, vpg=14 * A + one - 16) == 9
    assert append(lib, kp=15 * A) == 9 and append(lib, ks=17 * A) == 9 and append(lib, ks=14 * A) == 9
    assert append(lib, kp=2 * A) == 9 and append(lib, vs=13 * A) == 9
    assert append(lib, k=2 * A, v=2 * A) in REACH  # (both are only read)
    assert read(lib, k=14 * A) == 9 and read(lib, v=2 * A) == 9 and read(lib, k=16 * A) == 9 and read(lib, v=12 * A) == 9
    assert read(lib, kp=15 * A) in REACH
    assert paged(lib, out=14 * A) == 9 and paged(lib, lse=16 * A) == 9 and paged(lib, ws=17 * A) == 9
    assert paged(lib, out=A) == 9 and paged(lib, lse=5 * A) == 9


def test_workspace(lib):
    assert Q.evo_paged8_fwd_workspace_bytes(64, 2, 8, 2, 64, 10, 16, 4, 16) > 0
    few, long = (Q.evo_paged8_fwd_workspace_bytes(2, 2, 8, 2, 64, 10, 16, n, 16) for n in (64, 65))
    assert few == 0 and 0 < long < 1 << 23  # single tokens: 16 rows a piece, none where nothing is cut
    # many rows: a copy of what the table can hold, up to 512 MB
    room = [Q.evo_paged8_fwd_workspace_bytes(2000, 2, 8, 2, 64, 10, 16, n, 16) for n in (8, 1 << 15, (1 << 15) + 1)]
    assert room[1] >= 1 << 29 > room[2] and room[0] >= 4 * 2 * 128 * 2 * 64
    assert Q.evo_paged8_fwd_workspace_bytes(64, 2, 8, 2, 72, 10, 16, 4, 16) == 0
    assert Q.evo_paged8_fwd_workspace_bytes(64, 2, 8, 2, 64, 10, 16, 4, 32) == 0


def test_binding_refuses_on_cpu():
    """What the binding looks at before it asks for a device."""
    q, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales, lens, table = torch.ones(3, 2, 1), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        Q.evo_rotary(q, None, torch.zeros(4, dtype=torch.int32), torch.ones(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="q must be"):
        Q.evo_rotary(q.float(), None, torch.zeros(4, dtype=torch.int32), torch.ones(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        Q.evo_cache8_append(q, q, cu, lens, pages, pages, scales, scales, table)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        Q.evo_cache8_read(pages.view(torch.uint8), pages, scales, scales, cu, lens, table, 4)
    with pytest.raises(ValueError, match="dtype"):
        Q.evo_cache8_read(pages, pages, scales, scales, cu, lens, table, 4, torch.float32)
    with pytest.raises(ValueError, match="heads of"):
        Q.evo_paged8_fwd(q[:, :1, :32], pages, pages, scales, scales, cu, lens, table)
