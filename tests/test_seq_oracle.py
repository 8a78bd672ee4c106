"""The fp64 oracle of the causal-sequence operators against differences, a loop over
single scores, closed forms and invariants (CPU)."""
import math

import numpy as np
import pytest

from oracle import seq_oracle as O


def draw(seed, n, L, Hq, Hk, D):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in ((n, Hq, D), (L, Hk, D), (L, Hk, D), (n, Hq, D))]


def test_forward_against_single_scores():
    q, k, v, _ = draw(0, 3, 5, 4, 2, 8)
    o, lse, w, _ = O.attend(q, k, v, 0.3)
    for h in range(4):
        for i in range(3):
            e = [math.exp(0.3 * sum(q[i, h, d] * k[j, h // 2, d] for d in range(8))) for j in range(5 - 3 + i + 1)]
            assert abs(lse[h, i] - math.log(sum(e))) < 1e-12
            for d in range(8):
                assert abs(o[i, h, d] - sum(x / sum(e) * v[j, h // 2, d] for j, x in enumerate(e))) < 1e-12
    assert np.allclose(w.sum(1), 3 * 2)  # each row's weights sum to 1


def test_rows_that_see_nothing():
    """More new tokens than keys: the first rows are empty."""
    q, k, v, _ = draw(1, 4, 2, 1, 1, 8)
    o, lse, w, _ = O.attend(q, k, v, 1.0)
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[0, :2]))
    assert np.allclose(o[2, 0], v[0, 0]) and np.isclose(lse[0, 2], q[2, 0] @ k[0, 0])
    assert np.isclose(w.sum(), 2)


@pytest.mark.parametrize("Hq,Hk", [(2, 2), (4, 2), (3, 1)])
def test_gradients_against_differences(Hq, Hk):
    q, k, v, do = draw(2, 5, 5, Hq, Hk, 8)
    f = lambda: float(np.sum(O.attend(q, k, v, 0.4)[0] * do))
    g = O.gradients(q, k, v, do, 0.4)
    rng = np.random.default_rng(3)
    for x, dx in zip((q, k, v), g):
        for _ in range(12):
            i = tuple(rng.integers(0, s) for s in x.shape)
            old, step = x[i], 1e-5
            x[i] = old + step
            up = f()
            x[i] = old - step
            down = f()
            x[i] = old
            assert abs((up - down) / (2 * step) - dx[i]) < 1e-8


def test_choice():
    w = np.array([1.0, 5.0, np.nan, 5.0, 0.0, -0.0, 2.0, -np.inf])
    assert O.choose(w, 8, 8, 2) == list(range(8))
    assert O.choose(w, 8, 3, 1) == [1, 3, 7]
    assert O.choose(w, 8, 2, 1) == [1, 7]            # the older of two equal ones
    assert O.choose(w, 8, 2, 0) == [1, 3]
    assert O.choose(w, 8, 7, 0) == [0, 1, 3, 4, 5, 6, 7]  # the NaN goes first
    assert O.choose(w, 8, 4, 4) == [4, 5, 6, 7]
    assert O.choose(w, 6, 4, 0) == [0, 1, 3, 4]
