"""The attention mixer's and the cache's holders on the host: what they refuse and count.  No GPU needed: the
holders live on the CPU and no kernel is launched."""
import pytest
import torch

from mamba_ssm_layer_gb300 import abi, synth
from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache

bf = torch.bfloat16
DIMS = synth.TINY_ATTENTION
CALLS = ("w8a16_gemv", "m2_qk_norm_rope", "m2_kv4_append", "m2_kv4_gather", "m2_attn_prefill_varlen",
         "m2_attn_decode_kv4")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()


@pytest.fixture
def calls(monkeypatch):
    """Names and arguments of the entry points that a holder calls, in place of the calls."""
    seen = []
    for name in CALLS:
        monkeypatch.setattr(abi, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    return seen


@pytest.fixture(scope="module")
def mixer():
    return DeviceAttention(synth.make_attention(DIMS, 9), device="cpu")


class Stream:
    cuda_stream = 0


def prefill(m, cache, b, new, **over):
    a = dict(x=torch.zeros(sum(new), m.hidden, dtype=bf), row_pos=torch.zeros(sum(new), dtype=torch.int32),
             out=torch.zeros(sum(new), m.hidden, dtype=bf))
    a.update(over)
    m.prefill(a["x"], new, a["row_pos"], cache, 0, b, a["out"], Stream())


def decode(m, cache, b, **over):
    a = dict(x=torch.zeros(cache.nseq, m.hidden, dtype=bf), kv_len=cache.pos + 1,
             out=torch.zeros(cache.nseq, m.hidden, dtype=bf))
    a.update(over)
    m.decode(a["x"], cache, 0, b, a["kv_len"], a["out"], Stream())


def cache_of(m, nseq=2, **over):
    a = dict(n_layers=1, nseq=nseq, n_pages=12, max_tokens=256, n_kv_heads=m.Hkv, head_dim=m.D, device="cpu")
    a.update(over)
    return Kv4Cache(**a)


@pytest.mark.parametrize("new,over", [
    ([5, 8], {}),                                         # more rows than max_rows
    ([5], {}), ([1, 2, 3], {}), ([-1, 4], {}),            # not a count for every sequence
    ([3, 4], dict(x=torch.zeros(6, DIMS["hidden"], dtype=bf))),
    ([3, 4], dict(x=torch.zeros(8, DIMS["hidden"], dtype=bf))),
    ([3, 4], dict(x=torch.zeros(7, DIMS["hidden"] - 8, dtype=bf))),
    ([3, 4], dict(x=torch.zeros(7, DIMS["hidden"] + 8, dtype=bf)[:, 8:])),  # the rows are not dense
    ([3, 4], dict(x=torch.zeros(7, DIMS["hidden"]))),
    ([3, 4], dict(out=torch.zeros(6, DIMS["hidden"], dtype=bf))),
    ([3, 4], dict(row_pos=torch.zeros(6, dtype=torch.int32))),
    ([3, 4], dict(row_pos=torch.zeros(7, dtype=torch.int64)))])
def test_prefill_refuses_rows_that_do_not_fit(mixer, calls, new, over):
    cache, b = cache_of(mixer), mixer.buffers(12, 64, 2)
    prefill(mixer, cache, b, [3, 4])  # the call itself is fine
    assert len(calls) == 5
    with pytest.raises(abi.M2Error):
        prefill(mixer, cache, b, new, **over)
    assert len(calls) == 5  # refused before any launch


@pytest.mark.parametrize("max_keys,held,ok", [(0, [0, 0], True), (0, [1, 0], False), (27, [20, 0], True),
                                              (26, [20, 0], False), (26, [0, 20], False)])
def test_prefill_refuses_more_keys_than_its_buffer_holds(mixer, calls, max_keys, held, ok):
    cache, b = cache_of(mixer), mixer.buffers(12, max_keys, 2)
    cache.tokens[:] = held
    if ok:
        prefill(mixer, cache, b, [3, 4])
        assert [n for n, _ in calls].count("m2_kv4_gather") == (1 if any(held) else 0)
    else:
        with pytest.raises(abi.M2Error) as e:
            prefill(mixer, cache, b, [3, 4])
        assert e.value.status == abi.M2_ERR_WORKSPACE and not calls


@pytest.mark.parametrize("over", [
    dict(x=torch.zeros(3, DIMS["hidden"], dtype=bf)), dict(x=torch.zeros(1, DIMS["hidden"], dtype=bf)),
    dict(out=torch.zeros(1, DIMS["hidden"], dtype=bf)), dict(kv_len=torch.zeros(1, dtype=torch.int32)),
    dict(kv_len=torch.zeros(2, dtype=torch.int64))])
def test_decode_refuses_rows_that_do_not_fit(mixer, calls, over):
    cache, b = cache_of(mixer), mixer.buffers(12, 64, 2)
    decode(mixer, cache, b)
    assert len(calls) == 5
    with pytest.raises(abi.M2Error):
        decode(mixer, cache, b, **over)
    with pytest.raises(abi.M2Error):
        decode(mixer, cache, mixer.buffers(1, 64, 2))
    assert len(calls) == 5


def test_buffers_and_caches_of_other_heads_are_refused(mixer, calls):
    other = DeviceAttention(synth.make_attention(dict(DIMS, kv_heads=1), 9), device="cpu")
    with pytest.raises(abi.M2Error):
        prefill(mixer, cache_of(mixer), other.buffers(12, 64, 2), [3, 4])
    for heads in (dict(n_kv_heads=1), dict(head_dim=128)):
        with pytest.raises(abi.M2Error):
            prefill(mixer, cache_of(mixer, **heads), mixer.buffers(12, 64, 2), [3, 4])
        with pytest.raises(abi.M2Error):
            decode(mixer, cache_of(mixer, **heads), mixer.buffers(12, 64, 2))
    assert not calls


def test_cache_counts_what_a_captured_loop_advanced():
    c = Kv4Cache(1, 2, 20, 640, 2, 64, device="cpu")
    c.reserve([100, 70])
    c.advance([100, 70])
    for _ in range(40):  # as in a capture: the device counts, the host does not see it
        c.pos.add_(1)
    c.advance([40, 40], on_device=False)
    assert c.pos.tolist() == c.tokens == [140, 110]
    c.reserve([64, 64])
    assert (c.table >= 0).sum(1).tolist() == [4, 3]  # 204 and 174 tokens
    c.advance([64, 64])
    assert c.pos.tolist() == c.tokens == [204, 174]


@pytest.mark.parametrize("new,error", [([100, 193], RuntimeError), ([193, 10], RuntimeError), ([10], abi.M2Error),
                                       ([10, 10, 10], abi.M2Error), ([10, -1], abi.M2Error),
                                       ([190, 190], RuntimeError)])
def test_a_refused_reserve_hands_out_nothing(new, error):
    c = Kv4Cache(1, 2, 5, 192, 2, 64, device="cpu")
    c.reserve([5, 0])
    table = c.table.clone()
    with pytest.raises(error):
        c.reserve(new)
    assert torch.equal(c.table, table) and len(c._free) == 4
    with pytest.raises(abi.M2Error):
        c.advance([1])
    assert c.pos.tolist() == c.tokens == [0, 0]


@pytest.mark.parametrize("new,held,runs", [
    # runs: (first row, first key row, sequences, over the cache) of each call to attention
    ([3, 4], [0, 0], [(0, 0, 2, False)]),
    ([3, 4], [5, 6], [(0, 0, 2, True)]),
    ([3, 4], [0, 6], [(0, 0, 1, False), (3, 0, 1, True)]),
    ([3, 4, 2, 1], [5, 0, 0, 9], [(0, 0, 1, True), (3, 3, 2, False), (9, 8, 1, True)]),
    # sequences without new rows take part in neither
    ([0, 4, 0, 2], [50, 0, 7, 9], [(0, 0, 1, False), (4, 0, 1, True)]),
    ([0, 0], [4, 0], [])])
def test_a_first_prompt_attends_to_its_own_rows_whatever_the_batch(mixer, calls, new, held, runs):
    n = len(new)
    cache, b = cache_of(mixer, n), mixer.buffers(12, 24, n)
    cache.tokens[:] = held
    a = dict(x=torch.zeros(sum(new), mixer.hidden, dtype=bf), row_pos=torch.zeros(sum(new), dtype=torch.int32),
             out=torch.zeros(sum(new), mixer.hidden, dtype=bf))
    mixer.prefill(a["x"], new, a["row_pos"], cache, 0, b, a["out"], Stream(), first_over_cache=False)
    got = [x for name, x in calls if name == "m2_attn_prefill_varlen"]
    assert len(got) == len(runs)
    row = lambda t, base: (t.data_ptr() - base.data_ptr()) // (base.stride(0) * 2)  # noqa: E731
    for (q, _, k, ld_k, v, ld_v, out, _, *_, cu_q, cu_k, _, _), (q0, k0, count, over) in zip(got, runs):
        assert row(q, b["q"]) == row(out, b["attn"]) == q0 and len(cu_q) == count + 1
        assert row(k, b["keys"] if over else b["k"]) == k0
        assert row(v, b["keys"] if over else b["qkv"]) == k0
        assert (ld_k, ld_v) == ((2 * mixer.Hkv * mixer.D,) * 2 if over else (mixer.Hkv * mixer.D, mixer.n_qkv))
    gathers = [x for name, x in calls if name == "m2_kv4_gather"]
    want = [0]
    for m, t in zip(new, held):
        want.append(want[-1] + (m + t if m and t else 0))
    assert [list(x[5]) for x in gathers] == ([want] if want[-1] else [])


@pytest.mark.parametrize("held", [[0, 0], [0, 6], [3, 6]])
def test_every_prompt_over_the_cache(mixer, calls, held):
    cache, b = cache_of(mixer), mixer.buffers(12, 24, 2)
    cache.tokens[:] = held
    a = [torch.zeros(7, mixer.hidden, dtype=bf) for _ in range(2)]
    mixer.prefill(a[0], [3, 4], torch.zeros(7, dtype=torch.int32), cache, 0, b, a[1], Stream(), first_over_cache=True)
    names = [name for name, _ in calls]
    assert names.count("m2_attn_prefill_varlen") == names.count("m2_kv4_gather") == 1
    assert dict(calls)["m2_attn_prefill_varlen"][2].data_ptr() == b["keys"].data_ptr()


def test_cache_slot_without_a_sequence():
    c = Kv4Cache(1, 3, 9, 192, 2, 64, device="cpu")
    c.reserve([10, 70, 5])
    c.advance([10, 70, 5])
    c.release(1, idle=True)
    assert c.pos.tolist() == [10, abi.M2_KV4_IDLE, 5] and c.tokens == [10, 0, 5]
    c.pos.add_(1)  # a captured loop counts every slot
    c.advance([1, 0, 1], on_device=False)
    c.reserve([1, 0, 1])
    assert c.pos.tolist() == [11, abi.M2_KV4_IDLE + 1, 6]
    c.reserve([0, 100, 0])  # the slot's next sequence
    c.advance([0, 100, 0])
    assert c.pos.tolist() == c.tokens == [11, 100, 6]
