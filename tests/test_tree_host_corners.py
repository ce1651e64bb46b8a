"""Faults that were found in the holders and entry points for trees of drafted tokens, each held
by what it accepted or refused wrongly.  No GPU needed."""
import contextlib

import pytest
import torch

from mamba_ssm_layer_gb300 import abi, synth
from tests.test_tree_host import Stream, calls, ints  # noqa: F401

CU = [0, 3, 5]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()


def mixer(nseq=2):
    from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache
    m = DeviceAttention(synth.make_attention(synth.TINY_ATTENTION, 9), device="cpu")
    return m, Kv4Cache(2, nseq, 12, 256, m.Hkv, m.D, device="cpu")


def layer(nseq=2):
    from mamba_ssm_layer_gb300.layer import DeviceLayer
    dl = DeviceLayer(synth.make_layer(synth.TINY, synth.WL_TINY_DECODE), device="cpu")
    return dl, dl.new_state(nseq, device="cpu"), dl.workspace_tree(nseq, 5, device="cpu")


@pytest.mark.parametrize("count", [torch.arange(4, dtype=torch.int32).view(2, 2)[:, 0], ints(1).expand(2),
                                   torch.arange(4, dtype=torch.int32)[::2]])
def test_counts_lie_one_behind_the_other(calls, count):  # noqa: F811
    _, cache = mixer()
    dl, st, ws = layer()
    path = ints(0, 2, -1, 0, -1)
    with pytest.raises(abi.M2Error):
        cache.keep(CU, path, count, 0)
    with pytest.raises(abi.M2Error):
        dl.tree_commit(CU, path, count, st, ws, Stream())
    assert not calls and cache.pos.tolist() == [0, 0]


def test_a_count_of_another_shape_advances_the_cache(calls, monkeypatch):  # noqa: F811
    """It ended with an error after the rows had been moved."""
    from mamba_ssm_layer_gb300 import attention
    monkeypatch.setattr(attention, "_on", lambda stream: contextlib.nullcontext())
    _, cache = mixer()
    cache.keep(CU, ints(0, 2, -1, 0, -1), ints(2, 1).view(2, 1), 0)
    assert [n for n, _ in calls] == ["m2_kv4_keep"] * 2 and cache.pos.tolist() == [2, 1]
    assert cache.pos.shape == (2,)


WS_DIMS = [synth.NEMOTRON_H_8B, synth.TINY]


@pytest.mark.parametrize("dims", WS_DIMS)
def test_a_workspace_for_more_rows_holds_fewer(dims):
    """Whatever passes of up to so many rows need; the k-split partials are not monotone in the rows."""
    d = abi.dims_struct(dims)
    for size in (lambda t: abi.m2_workspace_bytes_tree(d, 128, t), lambda t: abi.m2_workspace_bytes_varlen(d, 8, t),
                 lambda t: abi.m2_workspace_bytes(d, 0, t)):
        sizes = [size(t) for t in range(1, 700)]
        assert sizes == sorted(sizes)
        assert size(20000) >= sizes[-1]


def test_a_layer_workspace_for_more_nodes_serves_fewer():
    """The workspace is looked at before hidden, which is missing here."""
    from tests.test_tree_host import FAKE, _layer
    d, M = abi.dims_struct(synth.NEMOTRON_H_8B), abi.M2_ERR_ARG
    for most in (129, 130, 156, 257, 320, 328):
        size = abi.m2_workspace_bytes_tree(d, 128, most)
        for n in range(most - 80, most + 1):
            cu = [0] + [n * (i + 1) // 128 for i in range(128)]
            st = abi.mamba2_layer_tree(d, _layer(), None, cu, FAKE, FAKE, FAKE, FAKE, FAKE, size, check=False)
            assert st == M, (most, n)


def test_arrays_by_sequence_are_checked_without_nodes():
    from tests.test_tree_host import COMMIT, FAKE, VERIFY
    for fn, base, by_seq in ((abi.mamba2_tree_commit, COMMIT, ("h", "conv_state", "conv_pos", "h_out", "conv_state_out",
                                                               "conv_pos_out", "A_log", "dt_bias", "count")),
                             (abi.m2_verify_tree, VERIFY, ("u_next", "count", "next_token"))):
        for name in by_seq:
            assert fn(**dict(base, cu_nodes=[0, 0, 0], **{name: None}), check=False) == abi.M2_ERR_ARG
            assert fn(**dict(base, cu_nodes=[0, 0, 0], **{name: FAKE + 1}), check=False) == abi.M2_ERR_ALIGN
    n = abi.m2_launch_count()
    none = dict(xbc=None, ld_xbc=0, u=None, ld_u=0, dt_raw=None, ld_dt=0, path=None, H=1, P=3, N=16, G=1)
    assert abi.mamba2_tree_commit(**dict(COMMIT, cu_nodes=[0, 0, 0], **none), check=False) == abi.M2_OK  # all in place
    assert abi.m2_launch_count() == n


def test_passes_without_nodes():
    """No mock: nothing is launched, and nothing is refused."""
    m, cache = mixer()
    dl, st, ws = layer()
    none = torch.empty(0, dtype=torch.int32)
    x = torch.empty(0, m.hidden, dtype=torch.bfloat16)
    n = abi.m2_launch_count()
    m.tree(x, [0, 0, 0], none, none, cache, 1, m.buffers(8, 0, 2, trees=True), torch.empty_like(x), Stream())
    dl.tree(torch.empty(0, 256, dtype=torch.int16), [0, 0, 0], none, st, ws, Stream())
    dl.tree_commit([0, 0, 0], none, ints(0, 0), st, ws, Stream())
    assert abi.m2_launch_count() == n
    with pytest.raises(abi.M2Error):
        m.tree(x, [0, 0], none, none, cache, 1, m.buffers(8, 0, 2, trees=True), torch.empty_like(x), Stream())


def test_conv_refuses_outputs_over_its_inputs():
    """Nodes read their ancestors' rows, so that in place others would read outputs."""
    from tests.test_tree_host import CONV, FAKE
    n = abi.m2_launch_count()
    for ld, C, T, off in ((640, 600, 8, 0), (640, 600, 8, 599), (640, 600, 8, 640), (640, 600, 8, -600), (640, 600, 8, 45),
                          (640, 600, 8, 7 * 640 + 599), (600, 600, 1, 599), (640, 640, 8, -7 * 640)):
        over = dict(CONV, x=FAKE + 20000, out=FAKE + 20000 + 2 * off, ld_x=ld, ld_o=ld, Cc=C, cu_nodes=[0, T])
        assert abi.mamba2_tree_conv(**over, check=False) == abi.M2_ERR_ARG
    assert abi.m2_launch_count() == n
