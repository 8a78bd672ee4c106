"""Index arithmetic of the causal-sequence kernels (csrc/evo_seq_index.h), compiled for the host:
the lengths at which 32 bits run out are far beyond what a test on a GPU can attend to."""
import ctypes
import subprocess

import pytest

from memory_efficient_biased_gb300 import build

SOURCE = """
#include "evo_seq_index.h"
extern "C" int first_row(int ahead, int TQ, int group) { return evo::first_row(ahead, TQ, group); }
extern "C" int tile_rows(int left, int TQ, int group) { return evo::tile_rows(left, TQ, group); }
extern "C" unsigned newest_phase(unsigned uses, unsigned slots, unsigned i) { return evo::newest_phase(uses, slots, i); }
"""
GROUPS = (1, 2, 3, 8, 96, 127, 128)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    (d / "index.cpp").write_text(SOURCE)
    # -fwrapv: a product that does not fit wraps, as on the device
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", build.CSRC, "-o", str(d / "index.so"),
                    str(d / "index.cpp")], check=True)
    return ctypes.CDLL(str(d / "index.so"))


def test_first_row(lib):
    """A tile's rows that see a key, for keys up to 2^31 tokens in front of the tile."""
    for G in GROUPS:
        TQ = 128 // G
        for ahead in [-(2 ** 31) + 1025, max(-(2 ** 31 // G) - 1, -(2 ** 31)), -(2 ** 31 // G), -(2 ** 25), -(2 ** 25) - 1, *range(-300, 256)]:
            got = lib.first_row(ahead, TQ, G)
            seen = [r >= got for r in range(TQ * G)]
            assert seen == [r // G >= ahead for r in range(TQ * G)], (G, ahead)


def test_tile_rows(lib):
    """A tile's rows in the sequence, for ends up to 2^31 tokens behind the tile: what lies behind them is
    cleared, so a count that is too small would clear rows of the sequence or what is not the tile's."""
    for G in GROUPS:
        TQ = 128 // G
        for left in [2 ** 31 - 1025, min(2 ** 31 // G + 1, 2 ** 31 - 1025), 2 ** 25, 2 ** 24 + 1, *range(1, 300)]:
            assert lib.tile_rows(left, TQ, G) == min(left, TQ) * G, (G, left)


def test_newest_phase(lib):
    """What a CTA waits for before it leaves: each slot's newest phase, and never one that was not begun."""
    for slots in (1, 2, 3, 4, 5, 10):
        phases = [-1] * slots
        for uses in range(1, 60):
            phases[(uses - 1) % slots] += 1
            for i in range(min(slots, uses)):
                assert lib.newest_phase(uses, slots, i) == phases[i], (uses, slots, i)
