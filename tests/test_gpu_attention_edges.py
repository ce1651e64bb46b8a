"""Prompt attention where its warps run far apart, against the 64-bit form with the
tolerances of test_gpu_attention.py."""
import math

import pytest

from mamba_ssm_layer_gb300 import abi
from tests.test_gpu_attention import run_prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(8, 8), (7, 7)])
def test_prefill_marked_values_of_items_that_leave_a_tile_empty(H, Hkv, D):
    """Every CTA takes an item of two tiles, then several of one, all with values that are not finite: the second
    tile's warps still add back the first item's while the others are items ahead."""
    lens = [256] * 20 + [64] * 108

    def plant(q, k, v, cu_q, cu_k):
        for i, n in enumerate(lens):
            at = cu_k[i]
            if n == 256:
                v[at + 100:at + 256, D - 1::D] = math.inf
                v[at + 130, 2::D] = math.nan
            else:
                v[at + 10 + i % 40, i % D::D] = -math.inf
    run_prefill(lens, lens, H, Hkv, D, fix=plant)
