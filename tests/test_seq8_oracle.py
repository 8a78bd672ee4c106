"""The oracle of rotary positions and of the 8-bit cache, pinned (CPU)."""
import numpy as np
import pytest
import torch

from memory_efficient_biased_gb300 import evo_seq as Q
from oracle import seq_oracle as O


def test_e4m3_against_its_definition_and_torch():
    assert O.E4M3[0] == 0 and O.E4M3[1] == 2.0 ** -9 and O.E4M3[8] == 2.0 ** -6 and O.E4M3[-1] == 448 and len(O.E4M3) == 127
    assert np.all(np.diff(O.E4M3) > 0)
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(codes[:127], O.E4M3)
    mid = (O.E4M3[1:] + O.E4M3[:-1]) / 2
    x = np.concatenate([O.E4M3, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.linspace(-448, 448, 9999)])
    x = x[np.abs(x) <= 448].astype(np.float32)
    np.testing.assert_array_equal(O.round_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(O.round_e4m3(np.nan))


def test_scale_is_the_least_that_fits():
    for most in (0.0, 1e-30, 2.0 ** -64, 1.0, 448.0, 448.0001, 65504.0, 3.3e38):
        s = O.scale8(most)
        assert most <= 448 * s and (s == 2.0 ** -64 or most > 224 * s) and np.log2(s) == int(np.log2(s))


def test_append_in_pieces():
    """Appending token by token ends at the scale of appending at once, and at most one more rounding
    off in the tokens that a larger one came behind."""
    rng = np.random.default_rng(0)
    new = rng.standard_normal((37, 8)) * np.exp(rng.standard_normal((37, 1)) * 2)
    at_once, by_one = (np.zeros((48, 8)), np.zeros(3)), (np.zeros((48, 8)), np.zeros(3))
    O.append8(*at_once, new, 0, 16)
    for i in range(37):
        O.append8(*by_one, new[i:i + 1], i, 16)
    np.testing.assert_array_equal(at_once[1], by_one[1])
    s = np.repeat(at_once[1], 16)[:37, None]
    # half a step at the final scale, 2^-10 of it at the least; half of one at an earlier, smaller scale
    bound = np.maximum(np.abs(new) * 2.0 ** -4, s * 2.0 ** -10)
    assert np.all(np.abs(at_once[0][:37] * s - new) <= bound)
    assert np.all(np.abs(by_one[0][:37] * s - new) <= 2 * bound)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    """Turning back undoes a turn; scores depend on the distance alone; a gradient is the inverse turn."""
    rng = np.random.default_rng(1)
    f = Q.rotary_frequencies(12)[0].numpy()
    x, y = rng.standard_normal((2, 5, 3, 20))
    pos = np.array([0, 1, 7, -4, 1000])
    t = O.rotate(x, pos, f, interleaved, 1.5)
    np.testing.assert_allclose(O.rotate(t, pos, f, interleaved, 1 / 1.5, True), x, atol=1e-12)
    np.testing.assert_array_equal(t[..., 12:], x[..., 12:])
    a = np.sum(O.rotate(x, pos, f, interleaved) * O.rotate(y, pos + 3, f, interleaved), -1)
    b = np.sum(O.rotate(x, pos + 50, f, interleaved) * O.rotate(y, pos + 53, f, interleaved), -1)
    np.testing.assert_allclose(a, b, atol=1e-10)
    # d<rotate(x), y>/dx by differences
    g = O.rotate(y, pos, f, interleaved, 1.5, True)
    for _ in range(20):
        i = tuple(rng.integers(0, n) for n in x.shape)
        d = np.zeros_like(x)
        d[i] = 1e-6
        up = np.sum((O.rotate(x + d, pos, f, interleaved, 1.5) - O.rotate(x - d, pos, f, interleaved, 1.5)) * y) / 2e-6
        assert abs(up - g[i]) < 1e-7
    # pair 1 of a head of two pairs at position 1, by hand
    f2 = np.array([1.0, 0.25])
    z = O.rotate(np.arange(1.0, 5.0).reshape(1, 1, 4), [1], f2, interleaved)[0, 0]
    c, s = np.cos(0.25), np.sin(0.25)
    if interleaved:
        np.testing.assert_allclose(z[2:], [3 * c - 4 * s, 4 * c + 3 * s])
    else:
        np.testing.assert_allclose(z[[1, 3]], [2 * c - 4 * s, 4 * c + 2 * s])


def test_frequencies():
    f, one = Q.rotary_frequencies(64)
    assert f.dtype == torch.float64 and one == 1.0 and f[0] == 1.0 and abs(float(f[-1]) - 10000.0 ** (-62 / 64)) < 1e-18
    lin, _ = Q.rotary_frequencies(64, scaling="linear", stretch=4.0)
    assert torch.equal(lin, f / 4)
    up, _ = Q.rotary_frequencies(64, scaling="base", stretch=4.0)
    assert up[0] == 1.0 and abs(float(up[-1] * 4 / f[-1]) - 1) < 1e-12
    parts, factor = Q.rotary_frequencies(64, scaling="parts", stretch=4.0, trained=4096)
    turns = 4096 * f / (2 * np.pi)
    assert torch.equal(parts[turns >= 32], f[turns >= 32]) and torch.allclose(parts[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    assert torch.all(parts <= f) and torch.all(parts >= f / 4 * (1 - 1e-15)) and abs(factor - (0.1 * np.log(4) + 1)) < 1e-15
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, scaling="linear", stretch=-1.0), dict(rotary_dim=8, scaling="parts", stretch=2.0),
                dict(rotary_dim=8, scaling="parts", stretch=2.0, trained=100, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            Q.rotary_frequencies(**bad)
