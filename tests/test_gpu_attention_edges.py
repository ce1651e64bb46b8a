"""The attention operators where work is cut, handed on and ordered: against the 64-bit
form with the tolerances of test_gpu_attention.py."""
import math

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from tests import attention_ref as ref
from tests.attention_cover import cover
from tests.test_gpu_attention import Cache, close, run_decode, run_prefill

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


@pytest.mark.parametrize("lens,H,Hkv,D", [([600, 520], 128, 1, 64), ([1100, 3, 90], 256, 2, 128), ([37, 41] * 64, 64, 1, 64),
                                          ([50] * 128, 192, 3, 128)])
def test_prefill_more_tile_pairs_than_are_sorted(lens, H, Hkv, D):
    """More than 512 pairs of tiles in a launch: handed out in their own order."""
    def plant(q, k, v, cu_q, cu_k):
        v[cu_k[1] - 20, 3] = math.inf
        v[cu_k[-1] - 2, D - 1] = math.nan
    run_prefill(lens, lens, H, Hkv, D, fix=plant)


# ------------------------------------------------------------------ no token lost or counted twice where work is cut

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,Hkv,every", [
    ([20000], 8, 1, False), ([40000], 8, 8, False), ([1, 40000, 77, 64 * 31], 4, 1, False), ([5000, 3], 32, 8, True),
    ([5000, 3, 4999], 16, 4, False), ([900] * 40, 32, 8, True), ([4096] * 5, 16, 16, True), ([700], 32, 8, True),
    ([2048], 24, 2, True), ([130, 2047, 1, 64, 65], 9, 1, False), ([8191], 40, 2, True)])
def test_decode_counts_every_token_once(lens, H, Hkv, every, D):
    def plant(k, v, cu):
        assert cover(v, cu, Hkv, D, 64, every) <= 64
    run_decode(lens, H, Hkv, D, fix=plant)
    run_decode(lens, H, Hkv, D, fix=plant, width=max(64, -(-max(lens) // 64) * 2))  # as wide as a serving cache's table


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k,H,Hkv,every", [
    ([1], [9000], 8, 2, False), ([70], [3333], 8, 2, True), ([300], [2500], 5, 1, False), ([16], [20000], 8, 2, False),
    ([1, 40, 0, 9], [1500, 4000, 17, 3], 4, 4, False), ([513], [513], 8, 2, True), ([1200], [1200], 4, 1, False)])
def test_prefill_counts_every_token_once(lens_q, lens_k, H, Hkv, every, D):
    run_prefill(lens_q, lens_k, H, Hkv, D, fix=lambda q, k, v, cu_q, cu_k: cover(v, cu_k, Hkv, D, 128, every))


# ------------------------------------------------------------------ streams

def test_operators_run_on_their_stream():
    """Inputs that a side stream makes behind a long kernel, with no other order than the stream's own."""
    H, K, D, n = 8, 2, 64, 200
    g = torch.Generator(device="cuda").manual_seed(2)
    made = [torch.randn(n, (H + 2 * K) * D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    qkv = torch.zeros_like(made[0])
    c = Cache([n], K, D, 1)
    pos, end = torch.arange(n, dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = torch.tensor(abi.m2_rope_steps(10000.0, D), dtype=torch.int64).cuda()
    ws = torch.empty(abi.m2_attn_decode_kv4_workspace_bytes(1, H, K, D), dtype=torch.uint8, device="cuda")
    q, k, kk, vv, o, o1 = (torch.zeros(r, w * D, dtype=torch.bfloat16, device="cuda")
                           for r, w in ((n, H), (n, K), (n, K), (n, K), (n, H), (1, H)))
    w = (H + 2 * K) * D

    def chain(source, s):
        with torch.cuda.stream(s):
            qkv.copy_(source)
        abi.m2_qk_norm_rope(qkv, w, qkv[:, H * D:], w, q, H * D, k, K * D, None, None, pos, steps, n, H, K, D, D, False,
                            1e-5, s)
        abi.m2_kv4_append(c.struct, k, K * D, qkv[:, (H + K) * D:], w, [0, n], zero, s)
        abi.m2_kv4_gather(c.struct, kk, K * D, vv, K * D, [0, n], s)
        abi.m2_attn_prefill_varlen(q, H * D, kk, K * D, vv, K * D, o, H * D, H, K, D, [0, n], [0, n], 0.1, s)
        abi.m2_attn_decode_kv4(c.struct, q[n - 1:], H * D, o1, H * D, H, end, 0.1, ws, ws.numel(), s)
        with torch.cuda.stream(s):
            return o.clone(), o1.clone()

    side = torch.cuda.Stream()
    torch.cuda._sleep(1)
    want = chain(made[0], torch.cuda.current_stream())
    torch.cuda.synchronize()
    chain(made[1], torch.cuda.current_stream())  # other rows everywhere
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = chain(made[0], side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and the rows are those of the 64-bit form
    rk, rv = ref.rounded_rows(k.view(n, K, D)), ref.rounded_rows(qkv[:, (H + K) * D:].reshape(n, K, D))
    out, size = ref.attend(q.view(n, H, D), rk, rv, 0.1)
    close(got[0].view(n, H, D), out, 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -15) * size + 1e-30)
    close(got[1].view(1, H, D), out[-1:], 2.0 ** -8 * out[-1:].abs() + (2.0 ** -11 + 2.0 ** -15) * size[-1:] + 1e-30)


# ------------------------------------------------------------------ scores that are all -Inf

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q,n_k", [(300, 300), (40, 3000)])
def test_rows_whose_scores_are_all_minus_infinity_are_zeros(n_q, n_k, D):
    H, K = 4, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(r, w * D, device="cuda", generator=g).to(torch.bfloat16)
               for r, w in ((n_q, H), (n_k, K), (n_k, K)))
    first = n_k - n_q + 10  # rows 0 .. 9 see only such keys
    q.view(n_q, H, D)[..., 0] = 1.0
    k.view(n_k, K, D)[:first, :, 0] = -math.inf
    out = torch.full((n_q, H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    abi.m2_attn_prefill_varlen(q, H * D, k, K * D, v, K * D, out, H * D, H, K, D, [0, n_q], [0, n_k], 0.1)
    assert bool((out[:10] == 0).all())
    want, size = ref.attend(q[10:].view(-1, H, D), k[first:].view(-1, K, D), v[first:].view(-1, K, D), 0.1)
    close(out[10:].view(-1, H, D), want, 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -15) * size + 1e-30)


@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_of_an_infinite_query(D):
    """Its scores are all -Inf (zeros) or hold a NaN or +Inf (NaN)."""
    def plant(k, v, cu):
        k.view(-1, 2, D)[:, 0, 3] = -2.0
        k.view(-1, 2, D)[:, 1, 3] = torch.where(torch.arange(len(k), device="cuda") % 3 > 0, 1.0, -1.0).to(k.dtype)
    r = run_decode([500], 4, 2, D, fix=plant)
    r["q"][0, 3::D] = math.inf
    r["call"]()
    out = r["out"].view(4, D)
    assert bool((out[:2] == 0).all()) and bool(out[2:].isnan().all())
