"""The barrier protocols of the 8-bit cache's attention kernels, explored on the CPU as tests/test_seq_protocol.py does
those of the 16-bit kernels (csrc/evo_seq8_few.cu, csrc/evo_seq8_tiles.cu), and what their rings rest on."""
import os
import re

import pytest

from memory_efficient_biased_gb300 import build
from tests.test_seq_protocol import Role, explore


def constant(name, source):
    text = open(os.path.join(build.CSRC, source)).read()
    return int(re.search(r"\b%s = (\d+)" % name, text).group(1))


def counted(roles, special):
    counts = {b: 1 for r in roles.values() for s in r.steps for b in [s[0]] + s[2] + s[3] if b}
    for b in counts:
        for start, n in special:
            if b.startswith(start):
                counts[b] = n
    return roles, counts


def few_roles(items, warps=3, groups=2, stages=3, descs=2, readers=1):
    """items: (tiles, rounds of joined rows).  A tile is `groups` times what a warp takes at a time, and the warps take
    them by turns (12, 8 and 6 stages in the kernel: as here a warp has 1.5 times as many turns as a tile)."""
    roles = {n: Role() for n in ["keys", "values", "scales", "q"] + [f"compute{w}" for w in range(warps)]}
    use = merges = 0
    for it, (tiles, rounds) in enumerate(items):
        d, b = it % descs, it % 2
        roles["keys"].wait(f"desc_empty{d}", it // descs - 1)
        roles["keys"].arrive(f"desc_full{d}")
        for n, r in roles.items():
            if n != "keys":
                r.wait(f"desc_full{d}", it // descs)
                r.arrive(f"desc_empty{d}")
        roles["q"].wait(f"q_empty{b}", it // 2 - 1)
        roles["q"].arrive(f"q_full{b}")
        for t in range(use, use + tiles):
            for n in ("keys", "values", "scales"):
                roles[n].wait(f"empty{t % stages}", t // stages - 1)
                roles[n].arrive(f"full{t % stages}")
        for w in range(warps):
            c = roles[f"compute{w}"]
            c.wait(f"q_full{b}", it // 2)
            for n in range(use * groups, (use + tiles) * groups):
                if n % warps == w:
                    t = n // groups
                    c.wait(f"full{t % stages}", t // stages)
                    c.arrive(f"empty{t % stages}")
            c.wait(None, 0)
            c.arrive(f"q_empty{b}")
            for m in range(merges, merges + rounds):
                c.wait("merge_empty", m - 1)
                c.arrive("merge_full")
                if w < readers:
                    c.wait("merge_full", m)
                    c.arrive("merge_empty")
        use += tiles
        merges += rounds
    return counted(roles, [("full", 3), ("empty", groups), ("desc_empty", warps + 3), ("q_empty", warps), ("merge_full", warps),
                           ("merge_empty", readers)])


@pytest.mark.parametrize("items", [[(2, 1)], [(1, 1), (1, 1)], [(1, 2), (2, 1)]])
def test_few(items):
    assert explore(*few_roles(items, warps=2 if len(items) > 1 else 3, groups=1 if len(items) > 1 else 2,
                              stages=2 if len(items) > 1 else 3)) > 100


def test_a_stage_is_always_or_never_a_warp_s():
    """A warp that waited for some phases of a stage's barrier only could take one for another."""
    f = "evo_seq8_few.cu"
    warps, keys, stages = (constant(n, f) for n in ("kWarps", "kKeys", "kStages"))
    groups = 128 // keys
    for w in range(warps):
        looked = {t for n in range(20 * warps * groups * stages) if n % warps == w for t in [n // groups]}
        last = max(looked) // stages - 1
        for st in range(stages):
            phases = [t // stages for t in sorted(looked) if t % stages == st and t // stages <= last]
            assert phases == list(range(last + 1)) or not phases, (w, st)


def tiles_roles(items, slots=3, scales=2, bf16=True):
    """items: (tiles of query tile 0, of query tile 1), or (tiles,) for one query tile, its key tiles by turns."""
    roles = {"producer": Role(), "walk": Role(), "widen": Role()}
    p, w, x = roles["producer"], roles["walk"], roles["widen"]
    queries, turn, use, n = [0, 0], 0, 0, 0
    plan = []
    for item in items:
        one, tiles = len(item) == 1, max(item)
        share = [list(range(g, tiles, 2)) for g in (0, 1)] if one else [list(range(t)) for t in item]
        plan.append((tiles, turn if one else None, share))
        for b in ([turn] if one else [0, 1]):
            p.wait(f"q_empty{b}", queries[b] - 1)
            p.arrive(f"q_full{b}")
            if bf16:
                x.wait(f"q_full{b}", queries[b])
                x.arrive(f"q_ready{b}")
            queries[b] += 1
        turn ^= one
        for _ in range(tiles):
            w.wait(f"scale_empty{n % scales}", n // scales - 1)
            w.arrive(f"scale_full{n % scales}")
            n += 1
            for _ in range(2):
                p.wait(f"raw_empty{use % slots}", use // slots - 1)
                p.arrive(f"raw_full{use % slots}")
                x.wait(f"raw_full{use % slots}", use // slots)
                x.wait(f"empty{use % slots}", use // slots - 1)
                x.arrive(f"full{use % slots}")
                x.arrive(f"raw_empty{use % slots}")
                use += 1
    for g in (0, 1):
        m = roles[f"mma{g}"] = Role()
        c = roles[f"softmax{g}"] = Role()
        n = u = own = turns = merges = 0
        queries = [0, 0]
        for tiles, buf, share in plan:
            mine, qb = share[g], g if buf is None else buf
            for b in ([0, 1] if buf is None else [buf]):
                m.wait(f"q_ready{b}" if bf16 else f"q_full{b}", queries[b])
                queries[b] += 1
            if buf is None:
                m.arrive(f"q_empty{g ^ 1}")
            if not mine:
                m.arrive(f"q_empty{qb}")
            both = 0 if buf is not None else len(share[g ^ 1])
            for j in range(tiles):
                uk, uv = 2 * n, 2 * n + 1
                m.wait(f"full{uk % slots}", uk // slots)
                c.wait(f"scale_full{n % scales}", n // scales)
                if j not in mine:
                    m.arrive(f"empty{uk % slots}")
                    m.wait(f"full{uv % slots}", uv // slots)
                    m.arrive(f"empty{uv % slots}")
                    c.arrive(f"scale_empty{n % scales}")
                else:
                    if u:
                        m.wait(f"pv_done{g}", u - 1)
                    m.commit(f"s_full{g}")
                    m.commit(f"empty{uk % slots}")
                    if j == mine[-1]:
                        m.commit(f"q_empty{qb}")
                    m.wait(f"full{uv % slots}", uv // slots)
                    if j == mine[0]:
                        m.wait(f"o_free{g}", own - 1)
                    m.wait(f"p_half{g}", u)
                    m.wait(f"p_full{g}", u)
                    m.commit(f"pv_done{g}")
                    m.commit(f"empty{uv % slots}")
                    c.wait(f"s_full{g}", u)
                    if j < both:
                        c.wait(f"turn{g}", turns - 1 + g)
                        turns += 1
                    c.arrive(f"p_half{g}")
                    if j < both:
                        c.wait(None, 0)
                        c.arrive(f"turn{g ^ 1}")
                    c.wait(None, 0)
                    c.arrive(f"p_full{g}")
                    c.arrive(f"scale_empty{n % scales}")
                    u += 1
                n += 1
            own += bool(mine)
            if mine:
                c.wait(f"pv_done{g}", u - 1)
            two = buf is not None and bool(share[1])
            if g and buf is not None:
                if two:
                    c.arrive("merge_full")
                continue
            if two:
                c.wait("merge_full", merges)
                merges += 1
            if mine:
                c.arrive(f"o_free{g}")
            if two:
                c.arrive("o_free1")
    return counted(roles, [("empty", 2), ("q_empty", 2), ("scale_empty", 2)])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("items", [[(1, 2)], [(3,)], [(1, 1), (1,)], [(1,), (2,)]])
def test_tiles(items, bf16):
    assert explore(*tiles_roles(items, bf16=bf16)) > 1000
