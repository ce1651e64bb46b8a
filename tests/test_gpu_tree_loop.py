"""Trees of drafted tokens through layers, mixers and a whole small stack, as a decode loop uses them."""
import random

import numpy as np
import pytest
import torch

from mamba_ssm_layer_gb300 import abi, synth
from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache
from mamba_ssm_layer_gb300.layer import DeviceLayer, bits_u16, to_dev
from oracle import oracle as orc
from tests import attention_ref
from tests import tree_ref as ref
from tests.helpers import (TOL_BF16, DecisionLog, _dd, _g_codes, _rup, _u16, bf16_to_f64, check_state_all_heads,
                           floored_rel_err)
from tests.test_gpu_attention import BF16, EVAL, F16, close, offsets
from tests.test_gpu_tree import ints, paths_of, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


def candidates(ws, cu, d, hidden_out, r5, g_f16):
    """The tree pass's rounding decisions by node row (tests/helpers.py)."""
    di, dx, n_in = _dd(d)
    T = cu[-1]
    wm = abi.m2_workspace_map(abi.dims_struct(d), abi.M2_WS_KIND_TREE, len(cu) - 1, cu)
    c = {"R3": _u16(ws, wm["zx"], T, _rup(n_in, 8))[:, :n_in].copy(), "R4": _u16(ws, wm["u"], T, dx).copy()}
    if r5:
        c["R5"], c["R6"] = _g_codes(ws, wm, T, di, slice(0, T), g_f16), hidden_out.copy()
    return c


@pytest.mark.parametrize("dims,fmt,lens,kind", [
    (synth.TINY, "fp8", [5, 3], "tree"), (synth.TINY, "fp8", [64, 1, 0, 17], "tree"), (synth.TINY, "bf16", [9, 9], "forest"),
    (synth.NEMOTRON_H_8B, "fp8", [6], "chain"), (synth.NEMOTRON_H_8B, "fp8", [9, 16], "tree")])
def test_layer(dims, fmt, lens, kind):
    """Every leaf's path against the oracle's steps, and the state after a committed path."""
    lay = synth.make_layer(dims, synth.WL_TINY_DECODE, in_fmt=fmt, out_fmt=fmt)
    d, n, key = lay["dims"], len(lens), (synth.WL_TINY_DECODE, 90)
    parents, cu = trees(lens, kind, 2), offsets(lens)
    if len(lens) == 4:
        parents[0][40] = -2  # a padded place
    dl, ol, log = DeviceLayer(lay), orc.OracleLayer(lay), DecisionLog()
    st = dl.new_state(n)
    # some context: a prompt of each
    warm = [4 + i for i in range(n)]
    wcu = offsets(warm)
    x0 = to_dev(synth.make_hidden(sum(warm), d["hidden"], *key, 7))
    dl.prefill_varlen(x0, wcu, st, dl.workspace_varlen(n, sum(warm)))
    torch.cuda.synchronize()
    before = st[0].cpu().numpy(), bits_u16(st[1]), st[2].cpu().numpy()
    hid = synth.make_hidden(cu[-1], d["hidden"], *key, 8)
    x, ws = to_dev(hid), dl.workspace_tree(n, cu[-1])
    dl.tree(x, cu, ints([p for t in parents for p in t]), st, ws)
    torch.cuda.synchronize()
    got = bits_u16(x)
    assert all(np.array_equal(a, b) for a, b in zip(before, (st[0].cpu().numpy(), bits_u16(st[1]), st[2].cpu().numpy())))
    cand = candidates(ws, cu, d, got, cu[-1] > 8, fmt == "fp8")

    def follow(i, path):
        state = [before[0][i].astype(np.float64), before[1][i].copy(), before[2][i:i + 1].copy()]
        if len(path):
            r = [cu[i] + k for k in path]
            out = hid[r].copy()
            log.add(ol.run_decided(out, *state, {k: np.ascontiguousarray(v[r]) for k, v in cand.items()}), (i, path))
            err = floored_rel_err(bf16_to_f64(got[r]), bf16_to_f64(out), axis=-1)
            assert err <= TOL_BF16, (i, path, err)
        return state
    for i, t in enumerate(parents):
        paths = ref.paths(t)
        leaves = [r for r in range(len(t)) if paths[r] and r not in t]
        for r in leaves if len(leaves) < 6 else leaves[::len(leaves) // 5]:
            follow(i, paths[r])
        for r in range(len(t)):
            if not paths[r]:  # not part of the tree: the row goes through unchanged
                assert np.array_equal(got[cu[i] + r], hid[cu[i] + r])
    picked, flat = paths_of(parents, random.Random(3))
    dl.tree_commit(cu, ints(flat), ints([len(p) for p in picked]), st, ws)
    torch.cuda.synchronize()
    h, ring, pos = st[0].cpu().numpy(), bits_u16(st[1]), st[2].cpu().numpy()
    for i, path in enumerate(picked):
        want = follow(i, path)
        check_state_all_heads(h[i], want[0])
        assert np.array_equal(ring[i], want[1]) and int(pos[i]) == int(want[2][0]) == warm[i] + len(path)
    log.check()


def test_mixer_nodes_and_kept_rows_are_the_single_tokens():
    """Two rounds of drafting: attention of every node against the 64-bit form on the cache's values; then the kept rows
    are bit for bit what single tokens would have appended."""
    m = DeviceAttention(synth.make_attention(synth.TINY_ATTENTION, 9))
    H, K, D, n = m.H, m.Hkv, m.D, 3
    lens = [7, 1, 30]
    cu, T = offsets(lens), sum(lens)
    cache = Kv4Cache(2, n, 40, 400, K, D)
    b = m.buffers(200, 600, n, trees=True)
    pre = [60, 3, 100]
    x = to_dev(synth.make_hidden(sum(pre), m.hidden, 9, 50)).view(torch.bfloat16)
    cache.reserve(pre)
    pos = torch.cat([torch.arange(k) for k in pre]).to(torch.int32).cuda()
    for layer in range(2):
        m.prefill(x, pre, pos, cache, layer, b, torch.empty_like(x))
    cache.advance(pre)
    held = [[], []], [[], []], [[], []]
    k0, v0 = b["k"][:sum(pre)].view(-1, K, D), b["qkv"][:sum(pre), (H + K) * D:].reshape(-1, K, D)
    pc = offsets(pre)
    held = [[attention_ref.rounded_rows(t[pc[i]:pc[i + 1]]) for t in (k0, v0)] for i in range(n)]
    for turn in range(2):
        parents = trees(lens, "tree", turn)
        depth = [len(p) - 1 for t in parents for p in ref.paths(t)]
        seq = torch.tensor([i for i, k in enumerate(lens) for _ in range(k)], device="cuda")
        x = to_dev(synth.make_hidden(T, m.hidden, 9, 60 + turn)).view(torch.bfloat16)
        out = torch.empty_like(x)
        row_pos = cache.pos[seq] + torch.tensor(depth, dtype=torch.int32, device="cuda")
        cache.reserve(lens)
        for layer in range(2):
            m.tree(x, cu, ints([p for t in parents for p in t]), row_pos, cache, layer, b, out)
        q, k = b["q"][:T].view(T, H, D), b["k"][:T].view(T, K, D)
        v = b["qkv"][:T, (H + K) * D:].reshape(T, K, D)
        kr, vr = attention_ref.rounded_rows(k), attention_ref.rounded_rows(v)
        for i in range(n):
            r = slice(cu[i], cu[i + 1])
            kk, vv = torch.cat([held[i][0], kr[r]]), torch.cat([held[i][1], vr[r]])
            want, size, total, score = ref.attend(q[r], kk, vv, m.scale, len(held[i][0]), parents[i])
            close(b["attn"][r].view(-1, H, D), want,
                  BF16 * want.abs() + (F16 + EVAL + 2.0 ** -19 * score) * size + 2.0 ** -32 * total + 1e-30)
        picked, flat = paths_of(parents, random.Random(turn))
        count = [len(p) for p in picked]
        cache.keep(cu, ints(flat), ints(count)[:n])
        cache.advance(count, on_device=False)
        for i, path in enumerate(picked):
            rows = [cu[i] + r for r in path]
            held[i] = [torch.cat([held[i][0], kr[rows]]), torch.cat([held[i][1], vr[rows]])]
        assert cache.pos.tolist() == cache.tokens == [len(h[0]) for h in held]
        at = offsets(cache.tokens)
        for layer in range(2):
            gk, gv = (torch.empty(at[-1], K * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            abi.m2_kv4_gather(cache.struct[layer], gk, K * D, gv, K * D, at)
            for i in range(n):
                assert torch.equal(gk[at[i]:at[i + 1]].to(ref.F).view(-1, K, D), held[i][0])
                assert torch.equal(gv[at[i]:at[i + 1]].to(ref.F).view(-1, K, D), held[i][1])


def test_example_runs():
    from examples import drafted_tokens
    assert drafted_tokens.main(wide=False, steps=6)
