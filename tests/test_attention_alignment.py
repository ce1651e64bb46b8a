"""Device pointers of the attention operators that are not aligned to their elements are refused: no GPU needed."""
import pytest

from mamba_ssm_layer_gb300 import abi

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_append_refuses_positions_that_are_not_aligned(off):
    c = abi.kv4_cache(FAKE, 10, 8, 128, FAKE, 2, 5)
    assert abi.m2_kv4_append(c, FAKE, 1024, FAKE, 1024, [0, 1, 2], FAKE + off, check=False) == abi.M2_ERR_ALIGN
    assert abi.m2_kv4_append(c, None, 1024, None, 1024, [0, 0, 0], FAKE + off, check=False) == abi.M2_OK  # no rows
