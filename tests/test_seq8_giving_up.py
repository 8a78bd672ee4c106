"""A CTA of csrc/evo_seq8_few.cu that gives up: on the CPU, where its warps may stand then, and that what it waits for before it
leaves does come; on the GPU, that such a call says so, soon, and leaves the next ones as they are."""
import time

import numpy as np
import pytest
import torch

from memory_efficient_biased_gb300 import evo_attn as E
from memory_efficient_biased_gb300 import evo_seq as Q
from tests import seq8_util as C
from tests import seq_util as S
from tests.test_seq8_protocol import few_roles

LOADERS = ("keys", "values", "scales")


def given_up(roles, counts):
    """Every set of arrivals at the barriers of the stages, by loader, that a CTA may end with when each of its roles may give up at
    any wait: {(arrivals of a loader at each stage, ...)}."""
    names, order = sorted(roles), sorted(counts)
    index = {b: i for i, b in enumerate(order)}
    progs = [[(None if b is None else index[b], k, [index[x] for x in a]) for b, k, a, _ in roles[n].steps] for n in names]
    start = tuple(0 for _ in names), frozenset(), tuple(0 for _ in order)
    seen, todo, ends = {start}, [start], set()
    while todo:
        pcs, stopped, arrived = todo.pop()
        out = []
        for r, p in enumerate(progs):
            if r in stopped or pcs[r] == len(p):
                continue
            bar, phase, arr = p[pcs[r]]
            if bar is not None:
                out.append((pcs, stopped | {r}, arrived))
            if bar is None or arrived[bar] // counts[order[bar]] >= phase + 1:
                a = list(arrived)
                for x in arr:
                    a[x] += 1
                out.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], stopped, tuple(a)))
        if not out:
            stages = [b for b in order if b.startswith("full")]
            ends.add(tuple(tuple(sum(s[2].count(b) for s in roles[n].steps[:pcs[names.index(n)]]) for b in stages) for n in LOADERS))
        for s in out:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return ends


def test_what_a_cta_that_gave_up_waits_for():
    """No loading warp is ever a whole phase of a stage in front of another: the arrivals that the later ones still owe complete the phase
    that the copies belong to, and none after it.  Without them there are phases that never end."""
    roles, counts = few_roles([(3, 1)], warps=2, groups=1, stages=2)
    ends = given_up(roles, counts)
    assert len(ends) > 20
    lag = [max(x) - min(x) for end in ends for x in zip(*end)]
    assert max(lag) == 1


@pytest.mark.gpu
def test_a_call_that_gives_up_ends_soon():
    """Thousands of sequences in front of the one with work: the other warps' first wait is longer than the least limit.  Either kernel
    gives up in some calls, takes less than the limit of its own copies, and leaves the GPU as it was."""
    rng = np.random.default_rng(5)
    B, Hq, Hk, D, ctx = 65535, 8, 2, 128, 9000
    cache = C.coded(rng, [ctx], 64, 64, Hk, D, *[lambda b, n: (C.O.round_e4m3(rng.standard_normal((n, Hk, D))), np.full((141, Hk), 0.25))] * 2)
    table = torch.zeros(B, cache.table.shape[1], dtype=torch.int32, device="cuda")
    table[-1] = cache.table[0]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = ctx
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    few = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    for tokens, heads in ((3, Hq), (300, 64)):  # (64 heads of 2: too many for few rows)
        q = S.normal(rng, tokens, heads, D, dtype=torch.bfloat16)
        few[-1] = tokens
        args = q.cuda(), *cache.args(), few, lens, table
        want = Q.evo_paged8_fwd(*args, wait_limit_ns=2 * 10 ** 9)
        torch.cuda.synchronize()
        gave_up = 0
        for _ in range(20):
            began = time.monotonic()
            Q.evo_paged8_fwd(*args, wait_limit_ns=1, status=status)
            took = int(status), time.monotonic() - began
            status.zero_()
            assert took[0] in (0, 8) and took[1] < 1.0, took
            gave_up += took[0] == 8
        assert gave_up, "no wait ran out"
        again = Q.evo_paged8_fwd(*args, status=status)
        assert int(status) == 0
        for x, y in zip(want, again):
            assert torch.equal(x, y)
        C.check_close(S.f64(q), *cache.rows(0, ctx), S.f64(again[0]), S.f64(again[1]), D ** -0.5, torch.bfloat16, heads == Hq)
    assert E.evo_attn_device_status() == 0
