"""What the checks of the 8-bit cache's attention would notice, on the CPU: the oracle's own result, with a tile of keys left out
or counted twice, does not pass."""
import numpy as np
import pytest
import torch

from oracle import seq_oracle as O
from tests import seq8_util as C


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("ctx", [131071, 30011, 9001])
def test_a_tile_too_few_or_too_many_is_noticed(ctx, few, dtype):
    rng = np.random.default_rng(ctx)
    D = 64
    k, v = C.flat_rows(rng, ctx, D)
    k, q = k * 2.0 ** -5, torch.from_numpy(rng.standard_normal((1, 1, D))).to(dtype).double().numpy()
    o, z, _, p = O.attend(q, k[:, None], v[:, None], D ** -0.5)
    bound, lse_bound = C.close_bounds(q, k[:, None], v[:, None], z, p, D ** -0.5, dtype, few)
    bound, w = bound[0, 0], p[0, 0]
    tiles = -(-ctx // 128)
    mass = np.add.reduceat(w, np.arange(0, ctx, 128))
    part = np.stack([w[t * 128:(t + 1) * 128] @ v[t * 128:(t + 1) * 128] for t in range(tiles)])
    for times in (-1.0, 1.0):
        total = 1.0 + times * mass
        out = (o[0, 0] + times * part) / total[:, None]
        assert np.all(np.abs(np.log(total)) > 2 * lse_bound[0, 0])
        assert np.all((np.abs(out - o[0, 0]) > 2 * bound).any(1))
        # a tile whose keys count, and whose values do not (or twice)
        assert np.all((np.abs(times * part) > 2 * bound).any(1))
