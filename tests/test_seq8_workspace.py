"""When attention over the 8-bit cache needs no workspace (CPU only): on both sides of what include/evo_seq.h states."""
import pytest

from memory_efficient_biased_gb300 import evo_seq as Q
from tests.test_seq8_host import cache, lib, paged  # noqa: F401
from tests.test_seq_host import REACH, shape


def need(tokens, seqs, Hq, Hk, places):
    return Q.evo_paged8_fwd_workspace_bytes(tokens, seqs, Hq, Hk, 64, 10, 16, places // 16, 16)


def test_no_workspace(lib):  # noqa: F811
    """Single tokens, 32 heads of 8: floor(16 / 4) = 4 tokens a block, (tokens / 4 + seqs) * 8 blocks."""
    assert need(1, 1, 32, 8, 1024) == 0 < need(1, 1, 32, 8, 1040)  # 10 blocks on any GPU's SMs
    assert need(64, 64, 32, 8, 1024) > 0                           # 640
    assert need(64, 64, 32, 8, 128) == 0 < need(64, 64, 32, 8, 144)
    assert need(8, 1, 32, 8, 128) == 0 < need(9, 1, 32, 8, 128)    # rows: 32 and 36
    assert need(1, 1, 17, 1, 128) > 0                              # group above 16


@pytest.mark.parametrize("tokens,places,null_will_do", [(1, 1024, True), (64, 1024, False), (64, 128, True)])
def test_null(lib, tokens, places, null_will_do):  # noqa: F811
    got = paged(lib, s=shape(T=tokens, B=tokens, Hq=32, Hk=8), c=cache(cols=places // 16), ws=None)
    assert got in REACH if null_will_do else got == 1
