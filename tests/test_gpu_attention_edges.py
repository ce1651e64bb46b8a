"""Prompt attention where its warps run far apart, against the 64-bit form with the
tolerances of test_gpu_attention.py."""
import math

import pytest
import torch

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


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_cut_along_the_keys_times_out_cleanly(D):
    """Few rows over many keys, with waits that give up at once: every CTA of a cluster still comes to its barriers,
    the status says so, and the same call computes correctly afterwards."""
    H, K, n_q, n_k = 8, 2, 16, 20000
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = (torch.randn(r, w * D, device="cuda", generator=g).to(torch.bfloat16)
               for r, w in ((n_q, H), (n_k, K), (n_k, K)))

    def run():
        out = torch.zeros(n_q, H * D, dtype=torch.bfloat16, device="cuda")
        abi.m2_attn_prefill_varlen(q, H * D, k, K * D, v, K * D, out, H * D, H, K, D, [0, n_q], [0, n_k], 0.1)
        return out, abi.m2_device_status(clear=True)

    first = run()  # the first launch of a kernel in a process starts its roles late
    assert first[1] == abi.M2_OK
    try:
        abi.m2_set_wait_limit(1)
        assert run()[1] == abi.M2_ERR_TIMEOUT
        abi.m2_set_wait_limit(900000)  # the same kernel, a limit that suffices
        again = run()
        assert again[1] == abi.M2_OK and torch.equal(first[0], again[0])
    finally:
        abi.m2_set_wait_limit(0)
    again = run()
    assert again[1] == abi.M2_OK and torch.equal(first[0], again[0])
