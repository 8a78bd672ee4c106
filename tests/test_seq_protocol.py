"""The barrier protocols of the causal-sequence kernels, explored on the CPU.

A wait by parity cannot tell a phase from the one two further on: whoever waits has to be sure to look while
its phase is the newest one that ended.  Each role of a kernel is written down here as the waits and arrivals of its
loop, in the order of the source (csrc/evo_seq_bwd.cu, evo_seq_weights.cu, evo_seq_fwd.cu), and every interleaving of the roles
over a few tiles is followed: no wait may find its phase passed by a later one, none may be let through by an
earlier phase of the same parity, and all roles end.  A barrier that several warps wait on or arrive at alike has two of them here
(a fast and a slow one).
"""
import os
import re

import pytest

from memory_efficient_biased_gb300 import build


class Role:
    """Steps (barrier, phase waited for or None, what follows the wait): arrivals, and commits, which arrive later."""

    def __init__(self):
        self.steps = []

    def wait(self, bar, phase):  # phase -1: a fresh barrier lets it through
        self.steps.append([bar, phase, [], []])

    def arrive(self, bar):
        if not self.steps:
            self.steps.append([None, 0, [], []])
        self.steps[-1][2].append(bar)

    def commit(self, bar):
        self.steps[-1][3].append(bar)


def explore(roles, counts):
    """Follows every interleaving; returns how many states there are, or raises with what went wrong."""
    order = sorted(counts)
    index = {b: i for i, b in enumerate(order)}
    need = [counts[b] for b in order]
    names = sorted(roles)
    progs = []
    for n in names:
        progs.append([(None if b is None else index[b], k, [index[x] for x in a], [index[x] for x in c])
                      for b, k, a, c in roles[n].steps])
    # a state: where every role is, how many commits of each are still to arrive (in order), arrivals at every barrier
    queues = [[x for s in p for x in s[3]] for p in progs]
    start = (tuple(0 for _ in progs), tuple((0, 0) for _ in progs), tuple(0 for _ in order))
    seen, todo = {start}, [start]
    while todo:
        pcs, commits, arrived = todo.pop()
        moved = False
        out = []
        for r, p in enumerate(progs):
            if pcs[r] < len(p):
                bar, phase, arr, com = p[pcs[r]]
                ok = True
                if bar is not None:
                    done = arrived[bar] // need[bar]
                    if done > phase + 1:
                        raise AssertionError(f"{names[r]} waits for phase {phase} of {order[bar]}, which has ended {done} phases")
                    ok = (done - phase - 1) % 2 == 0
                    if ok and done < phase + 1:
                        raise AssertionError(f"{names[r]} is let through to {order[bar]} phase {phase} after {done}")
                if ok:
                    a = list(arrived)
                    for x in arr:
                        a[x] += 1
                    c = commits[r]
                    out.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:],
                                commits[:r] + ((c[0] + len(com), c[1]),) + commits[r + 1:], tuple(a)))
            issued, landed = commits[r]
            if landed < issued:
                a = list(arrived)
                a[queues[r][landed]] += 1
                out.append((pcs, commits[:r] + ((issued, landed + 1),) + commits[r + 1:], tuple(a)))
        for s in out:
            moved = True
            if s not in seen:
                seen.add(s)
                todo.append(s)
        if not moved and any(pc < len(p) for pc, p in zip(pcs, progs)):
            raise AssertionError("stuck: " + ", ".join(f"{n} at {p[pc]}" for n, p, pc in zip(names, progs, pcs) if pc < len(p)))
    return len(seen)


def declared(name, source):
    """How many barriers `name` has in a kernel's Bars."""
    text = open(os.path.join(build.CSRC, source)).read()
    m = re.search(r"uint64_t [^;]*\b%s(?:\[(\d+)\])?[,;]" % name, text)
    return int(m.group(1) or 1)


def streamed(items, mma, compute):
    """What dK/dV and dQ have in common: the producer, and the walk's release of the streamed tiles."""
    roles = {"producer": Role(), "walk": Role(), "mma": mma(items)}
    n = 0
    for it, tiles in enumerate(items):
        for j in range(tiles):
            p, w = roles["producer"], roles["walk"]
            p.wait(f"a_empty{n % 3}", n // 3 - 1)
            p.arrive(f"a_full{n % 3}")
            if j == 0:
                p.wait("own_empty", it - 1)
                p.arrive("own_full")
            p.wait(f"b_empty{n % 2}", n // 2 - 1)
            p.arrive(f"b_full{n % 2}")
            w.wait(f"a_full{n % 3}", n // 3)
            w.wait(f"b_full{n % 2}", n // 2)
            w.arrive(f"ready{n % 4}")
            n += 1
    for i in range(2):
        roles[f"compute{i}"] = compute(items)
    counts = {b: 1 for r in roles.values() for s in r.steps for b in [s[0]] + s[2] + s[3] if b}
    for b in counts:
        if b.startswith(("p_ready", "dp_free", "ds_ready", "acc_free")):
            counts[b] = 2
    return roles, counts


def dq_roles(items, ds_barriers):
    ds = lambda n: (f"ds_ready{n % ds_barriers}", n // ds_barriers)

    def mma(items):
        m, n, gathers = Role(), 0, 0

        def issue_s(x):
            m.wait(f"ready{x % 4}", x // 4)
            m.wait(f"a_full{x % 3}", x // 3)
            if gathers:
                m.wait("second_done", gathers - 1)
            m.commit(f"s_full{x % 2}")

        def issue_dp(x):
            m.wait(f"b_full{x % 2}", x // 2)
            if x:
                m.wait("dp_free", x - 1)
            m.commit("dp_full")
            m.commit(f"b_empty{x % 2}")

        for it, tiles in enumerate(items):
            m.wait("own_full", it)
            issue_s(n)
            issue_dp(n)
            for j in range(tiles):
                if j + 1 < tiles:
                    issue_s(n + 1)
                    issue_dp(n + 1)
                m.wait(*ds(n))
                if j == 0:
                    m.wait("acc_free", it - 1)
                m.commit("second_done")
                m.commit(f"a_empty{n % 3}")
                gathers += 1
                n += 1
            m.commit("own_empty")
            m.commit("acc_full")
        return m

    def compute(items):
        c, n = Role(), 0
        for it, tiles in enumerate(items):
            for _ in range(tiles):
                c.wait(f"s_full{n % 2}", n // 2)
                c.wait("dp_full", n)
                c.arrive("dp_free")
                c.wait(None, 0)  # dS takes its time
                c.arrive(ds(n)[0])
                n += 1
            c.wait("acc_full", it)
            c.arrive("acc_free")
        return c

    return streamed(items, mma, compute)


def dkv_roles(items):
    def mma(items):
        m, n = Role(), 0

        def issue_s(x):
            m.wait(f"ready{x % 4}", x // 4)
            m.wait(f"a_full{x % 3}", x // 3)
            if x:
                m.wait("dp_free", x - 1)
            m.commit("s_full")

        def issue_dp(x):
            m.wait(f"b_full{x % 2}", x // 2)
            if x:
                m.wait("second_done", x - 1)
            m.commit("dp_full")

        for it, tiles in enumerate(items):
            m.wait("own_full", it)
            issue_s(n)
            issue_dp(n)
            for j in range(tiles):
                m.wait("p_ready", n)
                if j == 0:
                    m.wait("acc_free", it - 1)
                m.commit(f"b_empty{n % 2}")
                if j + 1 < tiles:
                    issue_s(n + 1)
                m.wait("ds_ready", n)
                m.commit("second_done")
                m.commit(f"a_empty{n % 3}")
                if j + 1 < tiles:
                    issue_dp(n + 1)
                n += 1
            m.commit("own_empty")
            m.commit("acc_full")
        return m

    def compute(items):
        c, n = Role(), 0
        for it, tiles in enumerate(items):
            for _ in range(tiles):
                c.wait("s_full", n)
                c.arrive("p_ready")
                c.wait("dp_full", n)
                c.arrive("dp_free")
                c.wait(None, 0)
                c.arrive("ds_ready")
                n += 1
            c.wait("acc_full", it)
            c.arrive("acc_free")
        return c

    return streamed(items, mma, compute)


def forward_roles(items, slots=5):
    """items: (tiles of query tile 0, of query tile 1), or (tiles,) for one query tile, its key tiles by turns."""
    roles = {"producer": Role(), "walk": Role()}
    p, w, use, queries, turn = roles["producer"], roles["walk"], 0, [0, 0], 0
    plan = []  # per item: key tiles, the query buffer of a single tile or None, key tiles of each warpgroup
    for item in items:
        one = len(item) == 1
        tiles = max(item)
        share = [list(range(g, tiles, 2)) for g in (0, 1)] if one else [list(range(t)) for t in item]
        plan.append((tiles, turn if one else None, share))
        for b in ([turn] if one else [0, 1]):
            p.wait(f"q_empty{b}", queries[b] - 1)
            p.arrive(f"q_full{b}")
            queries[b] += 1
        turn ^= one
        for _ in range(tiles):
            for kv in range(2):
                p.wait(f"empty{use % slots}", use // slots - 1)
                p.arrive(f"full{use % slots}")
                w.wait(f"full{use % slots}", use // slots)
                if kv:
                    w.arrive(f"v_ready{use // 2 % 8}")
                w.arrive(f"empty{use % slots}")
                use += 1
    for g in (0, 1):
        m = roles[f"mma{g}"] = Role()
        n = u = own = 0
        queries = [0, 0]
        for tiles, buf, share in plan:
            mine, qb = share[g], g if buf is None else buf
            for b in ([0, 1] if buf is None else [buf]):
                m.wait(f"q_full{b}", queries[b])
                queries[b] += 1
            if buf is None:
                m.arrive(f"q_empty{g ^ 1}")
            if not mine:
                m.arrive(f"q_empty{qb}")
            for j in range(tiles):
                uk, uv = 2 * n, 2 * n + 1
                m.wait(f"full{uk % slots}", uk // slots)
                if j not in mine:
                    m.arrive(f"empty{uk % slots}")
                    m.wait(f"v_ready{n % 8}", n // 8)
                    m.arrive(f"empty{uv % slots}")
                else:
                    if u:
                        m.wait(f"pv_done{g}", u - 1)
                    m.commit(f"s_full{g}")
                    m.commit(f"empty{uk % slots}")
                    if j == mine[-1]:
                        m.commit(f"q_empty{qb}")
                    m.wait(f"v_ready{n % 8}", n // 8)
                    m.wait(f"full{uv % slots}", uv // slots)
                    if j == mine[0]:
                        m.wait(f"o_free{g}", own - 1)
                    m.wait(f"p_half{g}", u)
                    m.wait(f"p_full{g}", u)
                    m.commit(f"pv_done{g}")
                    m.commit(f"empty{uv % slots}")
                    u += 1
                n += 1
            own += bool(mine)
        for warp in range(2):
            c = roles[f"softmax{g}{warp}"] = Role()
            u = turns = merges = 0
            for tiles, buf, share in plan:
                both = 0 if buf is not None else len(share[g ^ 1])
                for j in share[g]:
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
                    u += 1
                if share[g]:
                    c.wait(f"pv_done{g}", u - 1)
                two = buf is not None and bool(share[1])
                if g and buf is not None:
                    if two:
                        c.arrive("merge_full")
                    continue
                if two:
                    c.wait("merge_full", merges)
                    merges += 1
                if share[g]:
                    c.arrive(f"o_free{g}")
                if two:
                    c.arrive("o_free1")
    counts = {b: 1 for r in roles.values() for s in r.steps for b in [s[0]] + s[2] + s[3] if b}
    for b in counts:
        if b.startswith("empty"):
            counts[b] = 3
        elif b.startswith(("q_empty", "p_half", "p_full", "turn", "o_free", "merge_full")):
            counts[b] = 2
    return roles, counts


def weights_roles(items):
    roles = {"producer": Role(), "rows": Role(), "mma": Role()}
    p, r, m, n = roles["producer"], roles["rows"], roles["mma"], 0
    for it, tiles in enumerate(items):
        p.wait(f"k_empty{it % 2}", it // 2 - 1)
        p.arrive(f"k_full{it % 2}")
        m.wait(f"k_full{it % 2}", it // 2)
        for _ in range(tiles):
            p.wait(f"q_empty{n % 4}", n // 4 - 1)
            p.arrive(f"q_full{n % 4}")
            r.wait(f"rows_empty{n % 2}", n // 2 - 1)
            r.arrive(f"rows_full{n % 2}")
            m.wait(f"q_full{n % 4}", n // 4)
            m.wait(f"s_free{n % 2}", n // 2 - 1)
            m.commit(f"s_full{n % 2}")
            m.commit(f"q_empty{n % 4}")
            n += 1
        m.commit(f"k_empty{it % 2}")
    for g in (0, 1):
        for warp in range(2):
            c, n = roles.setdefault(f"compute{g}{warp}", Role()), 0
            for it, tiles in enumerate(items):
                for _ in range(tiles):
                    c.wait(f"rows_full{n % 2}", n // 2)
                    c.wait(f"s_full{n % 2}", n // 2)
                    c.arrive(f"s_free{n % 2}")
                    c.wait(None, 0)
                    c.arrive(f"rows_empty{n % 2}")
                    n += 1
                if g:
                    c.wait("half_free", it - 1)
                    c.arrive("half_full")
                else:
                    c.wait("half_full", it)
                    c.arrive("half_free")
    counts = {b: 1 for x in roles.values() for s in x.steps for b in [s[0]] + s[2] + s[3] if b}
    for b in counts:
        if b.startswith(("s_free", "rows_empty")):
            counts[b] = 4
        elif b.startswith("half"):
            counts[b] = 2
    return roles, counts


@pytest.mark.parametrize("items", [[4], [9], [1, 1, 2], [2, 3], [3, 1, 1], [5, 1, 4], [1] * 6])
def test_backward(items):
    """Items of so many tiles one behind the other, in each phase."""
    assert explore(*dkv_roles(items)) > 100
    assert explore(*dq_roles(items, declared("ds_ready", "evo_seq_bwd.cu"))) > 100


def test_a_phase_that_another_passes_is_found():
    """With one barrier for dS, dS of the next tile may be complete before the MMA warp looked for this one's."""
    with pytest.raises(AssertionError, match="ds_ready"):
        explore(*dq_roles([4], 1))


@pytest.mark.parametrize("items", [[(1, 2)], [(3,)], [(1, 1), (1,)], [(1,), (2,)]])
def test_forward(items):
    assert explore(*forward_roles(items)) > 1000


def test_weights():
    assert explore(*weights_roles([1, 1, 2])) > 1000
