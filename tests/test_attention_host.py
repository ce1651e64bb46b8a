"""The attention operators' refusals and host helpers: no GPU needed."""
import ctypes as C
import math

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from tests import attention_ref as ref

FAKE = 1 << 20  # a 16-byte-aligned non-null "device" address; never dereferenced
A = abi.M2_ERR_ARG
U = abi.M2_ERR_UNSUPPORTED
L = abi.M2_ERR_ALIGN


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    n = abi.m2_launch_count()
    yield
    assert abi.m2_launch_count() == n  # nothing below launches


def rope(**over):
    a = dict(q=FAKE, ld_q=4096, k=FAKE, ld_k=1024, q_out=FAKE, ld_qo=4096, k_out=FAKE, ld_ko=1024, q_w=FAKE, k_w=FAKE,
             pos=FAKE, rope_step=FAKE, T=3, H=32, Hkv=8, head_dim=128, rot_dim=128, interleaved=False, eps=1e-5)
    a.update(over)
    return abi.m2_qk_norm_rope(**a, check=False)


@pytest.mark.parametrize("over,want", [
    (dict(q=None), A), (dict(k=None), A), (dict(q_out=None), A), (dict(k_out=None), A), (dict(T=-1), A),
    (dict(H=0), A), (dict(Hkv=0), A), (dict(H=30), A), (dict(ld_q=4088), A), (dict(ld_ko=1016), A),
    (dict(pos=None), A), (dict(rope_step=None), A), (dict(rot_dim=-16), A), (dict(eps=-1.0), A),
    (dict(eps=math.nan), A), (dict(head_dim=96, rot_dim=64), U), (dict(rot_dim=24), U), (dict(rot_dim=144), U),
    (dict(q=FAKE + 2), L), (dict(k_out=FAKE + 8), L), (dict(ld_q=4100), L), (dict(q_w=FAKE + 4), L),
    (dict(pos=FAKE + 2), L), (dict(rope_step=FAKE + 4), L),
    (dict(T=0), abi.M2_OK),  # no rows: nothing to do
])
def test_rope_refuses(over, want):
    assert rope(**over) == want


def cache(**over):
    a = dict(pages=FAKE, n_pages=10, n_kv_heads=8, head_dim=128, block_table=FAKE, nseq=2, ld_table=5)
    a.update(over)
    return abi.kv4_cache(**a)


CACHE_REFUSALS = [(dict(pages=None), A), (dict(n_pages=0), A), (dict(n_kv_heads=0), A), (dict(head_dim=0), A),
                  (dict(head_dim=80), U), (dict(block_table=None), A), (dict(ld_table=0), A), (dict(ld_table=1 << 26), A),
                  (dict(pages=FAKE + 8), L), (dict(block_table=FAKE + 2), L)]


@pytest.mark.parametrize("fn", ["append", "gather"])
@pytest.mark.parametrize("over,want", [(dict(cache=o), w) for o, w in CACHE_REFUSALS] + [
    (dict(k=None), A), (dict(v=None), A), (dict(ld_k=1016), A), (dict(ld_v=1028), L), (dict(k=FAKE + 2), L),
    (dict(cu=[1, 2, 3]), A), (dict(cu=[0, 3, 2]), A), (dict(cu=[0, 3]), A), (dict(cu=[0, 0, 0]), abi.M2_OK)])
def test_cache_rows_refuse(fn, over, want):
    a = dict(cache={}, k=FAKE, ld_k=1024, v=FAKE, ld_v=1024, cu=[0, 2, 5])
    a.update(over)
    c = cache(**a["cache"])
    if fn == "append":
        st = lambda: abi.m2_kv4_append(c, a["k"], a["ld_k"], a["v"], a["ld_v"], a["cu"], FAKE, check=False)  # noqa: E731
    else:
        st = lambda: abi.m2_kv4_gather(c, a["k"], a["ld_k"], a["v"], a["ld_v"], a["cu"], check=False)  # noqa: E731
    if len(a["cu"]) != 3:
        with pytest.raises(abi.M2Error):
            st()
    else:
        assert st() == want


def test_append_needs_positions():
    assert abi.m2_kv4_append(cache(), FAKE, 1024, FAKE, 1024, [0, 1, 2], None, check=False) == A


@pytest.mark.parametrize("over,want", [
    (dict(q=None), A), (dict(k=None), A), (dict(v=None), A), (dict(out=None), A), (dict(H=31), A), (dict(Hkv=0), A),
    (dict(head_dim=256), U), (dict(ld_o=4088), A), (dict(ld_v=1020), A), (dict(ld_v=1028), L), (dict(out=FAKE + 8), L),
    (dict(cu_q=[0, 5, 4]), A), (dict(cu_k=[2, 5, 9]), A), (dict(scale=math.inf), A), (dict(scale=math.nan), A),
    (dict(cu_q=[0, 0, 0]), abi.M2_OK)])
def test_prefill_refuses(over, want):
    a = dict(q=FAKE, ld_q=4096, k=FAKE, ld_k=1024, v=FAKE, ld_v=1024, out=FAKE, ld_o=4096, H=32, Hkv=8, head_dim=128,
             cu_q=[0, 4, 9], cu_k=[0, 4, 9], scale=0.1)
    a.update(over)
    assert abi.m2_attn_prefill_varlen(**a, check=False) == want


def test_prefill_needs_matching_offsets():
    with pytest.raises(abi.M2Error):
        abi.m2_attn_prefill_varlen(FAKE, 4096, FAKE, 1024, FAKE, 1024, FAKE, 4096, 32, 8, 128, [0, 4, 9], [0, 9], 0.1)


@pytest.mark.parametrize("over,want", [(dict(cache=o), w) for o, w in CACHE_REFUSALS] + [
    (dict(q=None), A), (dict(out=None), A), (dict(H=12), A), (dict(H=0), A), (dict(kv_len=None), A),
    (dict(kv_len=FAKE + 2), L), (dict(ld_q=4092), A), (dict(ld_q=4100), L), (dict(q=FAKE + 2), L),
    (dict(scale=math.nan), A), (dict(ws=None), abi.M2_ERR_WORKSPACE), (dict(ws=FAKE + 16), abi.M2_ERR_WORKSPACE),
    (dict(ws_bytes=-1), abi.M2_ERR_WORKSPACE)])
def test_decode_refuses(over, want):
    a = dict(q=FAKE, ld_q=4096, out=FAKE, ld_o=4096, H=32, kv_len=FAKE, scale=0.1, ws=FAKE,
             ws_bytes=abi.m2_attn_decode_kv4_workspace_bytes(2, 32, 8, 128))
    over = dict(over)
    c = cache(**over.pop("cache", {}))
    a.update(over)
    if a["ws_bytes"] == -1:
        a["ws_bytes"] = abi.m2_attn_decode_kv4_workspace_bytes(2, 32, 8, 128) - 1
    assert abi.m2_attn_decode_kv4(c, **a, check=False) == want


def test_sizes():
    assert abi.m2_kv4_page_bytes(8, 128) == 8 * 72 * 128 and abi.m2_kv4_page_bytes(2, 64) == 2 * 72 * 64
    assert abi.m2_kv4_page_bytes(8, 80) == 0 and abi.m2_kv4_page_bytes(0, 128) == 0
    assert abi.m2_attn_decode_kv4_workspace_bytes(0, 32, 8, 128) == 0
    assert abi.m2_attn_decode_kv4_workspace_bytes(2, 30, 8, 128) == 0
    assert C.sizeof(abi.M2Kv4Cache) == 40  # the C struct's layout on a 64-bit host


def test_rope_steps():
    steps = abi.m2_rope_steps(10000.0, 128)
    assert len(steps) == 64
    for i, s in enumerate(steps):
        # a double's relative rounding in pow and the division
        assert math.isclose(s / 2.0 ** 64, 10000.0 ** (-2.0 * i / 128) / (2 * math.pi), rel_tol=1e-14)
    for bad in [(0.5, 128), (math.nan, 128), (10000.0, 20), (10000.0, 0), (10000.0, 144)]:
        with pytest.raises(abi.M2Error):
            abi.m2_rope_steps(*bad)


def test_reference_quantizer():
    """The 64-bit form itself: every level at every scale comes back, ties go to the even code."""
    lev = torch.tensor(ref.LEVELS + tuple(-v for v in ref.LEVELS), dtype=ref.F)
    for byte in (8, 9, 100, 127, ref.TOP_BYTE):
        x = lev * ref.SCALES[byte]
        code, b = ref.quantize(x)
        assert int(b) == byte and torch.equal(ref.dequantize(code, b), x)
    x = torch.zeros(16, dtype=ref.F)
    x[0] = 6.0
    x[1:8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert ref.rounded_rows(x)[1:8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
