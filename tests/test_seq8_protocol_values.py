"""The barrier protocol of csrc/evo_seq8_tiles.cu with fp16, where the warps that widen take a factor of every tile of values from the
ring of scales, and with bf16, where q is read as it arrives: explored on the CPU like tests/test_seq8_protocol.py."""
import pytest

from tests.test_seq_protocol import explore
from tests.test_seq8_protocol import tiles_roles


def roles(items, fp16, scales=2):
    r, counts = tiles_roles(items, scales=scales, bf16=False)
    if fp16:
        w, raw, n = [], 0, 0
        for step in r["widen"].steps:
            if step[0] and step[0].startswith("raw_full"):
                raw += 1
                if raw % 2 == 0:  # a tile of values
                    w.append([f"scale_full{n % scales}", n // scales, [f"scale_empty{n % scales}"], []])
                    n += 1
            w.append(step)
        r["widen"].steps = w
        for b in counts:
            if b.startswith("scale_empty"):
                counts[b] = 3
    return r, counts


@pytest.mark.parametrize("fp16", [True, False])
@pytest.mark.parametrize("items", [[(1, 2)], [(3,)], [(1, 1), (1,)], [(1,), (2,)]])
def test_tiles(items, fp16):
    assert explore(*roles(items, fp16)) > 1000
