"""Trees of drafted tokens: refusals of the entry points and the plain forms themselves.  No GPU needed."""
import math
import random

import pytest
import torch

from mamba_ssm_layer_gb300 import abi, synth
from tests import tree_ref as ref
from tests.test_attention_host import CACHE_REFUSALS, cache

FAKE = 1 << 20  # a 16-byte-aligned non-null "device" address; never dereferenced
A, U, L, W, OK = abi.M2_ERR_ARG, abi.M2_ERR_UNSUPPORTED, abi.M2_ERR_ALIGN, abi.M2_ERR_WORKSPACE, abi.M2_OK
TREES = [(dict(cu_nodes=[1, 2, 3]), A), (dict(cu_nodes=[0, 3, 2]), A), (dict(cu_nodes=[0, 65, 66]), U),
         (dict(cu_nodes=[0, 64, 128]), None), (dict(cu_nodes=[0, 0, 0]), OK)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    n = abi.m2_launch_count()
    yield
    assert abi.m2_launch_count() == n  # nothing below launches


def refused(fn, base, over, want, *first):
    a = dict(base)
    a.update(over)
    if want is not None:  # (None: the sizes are fine; here only other arguments could refuse, so nothing is called)
        assert fn(*first, **a, check=False) == want


CONV = dict(conv_state=FAKE, conv_pos=FAKE, x=FAKE, ld_x=640, w=FAKE, bias=FAKE, out=FAKE, ld_o=640, cu_nodes=[0, 3, 8],
            parent=FAKE, Cc=600, d_conv=4)


@pytest.mark.parametrize("over,want", TREES + [
    (dict(conv_state=None), A), (dict(conv_pos=None), A), (dict(x=None), A), (dict(w=None), A), (dict(out=None), A),
    (dict(parent=None), A), (dict(ld_x=599), A), (dict(ld_o=599), A), (dict(Cc=0), A), (dict(Cc=1 << 28), A),
    (dict(d_conv=1), U), (dict(d_conv=9), U), (dict(parent=FAKE + 2), L), (dict(conv_pos=FAKE + 2), L),
    (dict(x=FAKE + 1), L)])
def test_conv_refuses(over, want):
    refused(abi.mamba2_tree_conv, CONV, over, want)


SSM = dict(h=FAKE, x=FAKE, Bm=FAKE, Cm=FAKE, ld_in=10240, dt_raw=FAKE, ld_dt=18560, A_log=FAKE, D=FAKE, dt_bias=FAKE,
           y=FAKE, cu_nodes=[0, 3, 8], parent=FAKE, H=128, P=64, N=128, G=8)


@pytest.mark.parametrize("over,want", TREES + [(dict([(k, None)]), A) for k, v in SSM.items() if v == FAKE] + [
    (dict(ld_in=10242), A), (dict(ld_in=8188), A), (dict(ld_dt=127), A), (dict(H=0), A), (dict(G=3), A), (dict(N=48), U),
    (dict(P=257), U), (dict(h=FAKE + 8), L), (dict(Bm=FAKE + 4), L), (dict(y=FAKE + 4), L), (dict(A_log=FAKE + 2), L),
    (dict(H=1 << 21, ld_in=1 << 30, ld_dt=1 << 30, G=1, P=256), U)])
def test_ssm_refuses(over, want):
    refused(abi.mamba2_tree_ssm, SSM, over, want)


COMMIT = dict(h=FAKE, conv_state=FAKE, conv_pos=FAKE, h_out=FAKE, conv_state_out=FAKE, conv_pos_out=FAKE, xbc=FAKE,
              ld_xbc=18560, u=FAKE, ld_u=10240, dt_raw=FAKE, ld_dt=18560, A_log=FAKE, dt_bias=FAKE, cu_nodes=[0, 3, 8],
              path=FAKE, count=FAKE, H=128, P=64, N=128, G=8, d_conv=4)


@pytest.mark.parametrize("over,want", TREES[:-1] + [(dict([(k, None)]), A) for k, v in COMMIT.items() if v == FAKE] + [
    (dict(ld_xbc=10239), A), (dict(ld_u=10236), A), (dict(ld_u=10242), A), (dict(ld_dt=127), A), (dict(N=8), U),
    (dict(d_conv=9), U), (dict(h_out=FAKE + 4), L), (dict(count=FAKE + 2), L), (dict(u=FAKE + 2), L)])
def test_commit_refuses(over, want):
    refused(abi.mamba2_tree_commit, COMMIT, over, want)


VERIFY = dict(p=FAKE, ld_p=1000, q=FAKE, ld_q=1000, fmt=abi.M2_PROB_F32, V=1000, cu_nodes=[0, 3, 8], parent=FAKE,
              token=FAKE, u=FAKE, u_next=FAKE, path=FAKE, count=FAKE, next_token=FAKE)


@pytest.mark.parametrize("over,want", TREES[:-1] + [(dict([(k, None)]), A) for k, v in VERIFY.items() if v == FAKE and k != "q"]
                         + [(dict(fmt=3), abi.M2_ERR_FORMAT), (dict(V=0), A), (dict(V=(1 << 30) + 1), A),
                            (dict(ld_p=999), A), (dict(ld_q=999), A), (dict(p=FAKE + 2), L), (dict(q=FAKE + 2), L),
                            (dict(p=FAKE + 1, fmt=abi.M2_PROB_BF16), L), (dict(token=FAKE + 2), L)])
def test_verify_refuses(over, want):
    refused(abi.m2_verify_tree, VERIFY, over, want)


KEEP = dict(cu_nodes=[0, 3, 8], path=FAKE, count=FAKE, kv_pos=FAKE)


@pytest.mark.parametrize("over,want", [(dict(cache=o), w) for o, w in CACHE_REFUSALS] + TREES + [
    (dict(path=None), A), (dict(count=None), A), (dict(kv_pos=None), A), (dict(path=FAKE + 2), L)])
def test_keep_refuses(over, want):
    over = dict(over)
    c = cache(**over.pop("cache", {}))
    refused(abi.m2_kv4_keep, KEEP, over, want, c)


@pytest.mark.parametrize("over,want", [(dict(cache=o), w) for o, w in CACHE_REFUSALS] + TREES + [
    (dict(q=None), A), (dict(out=None), A), (dict(H=12), A), (dict(H=0), A), (dict(parent=None), A),
    (dict(kv_pos=None), A), (dict(kv_pos=FAKE + 2), L), (dict(ld_q=4092), A), (dict(ld_q=4100), L),
    (dict(out=FAKE + 2), L), (dict(scale=math.inf), A), (dict(ws=None), W), (dict(ws=FAKE + 16), W),
    (dict(ws_bytes=-1), W), (dict(cache=dict(ld_table=1 << 24)), U)])
def test_attention_refuses(over, want):
    over = dict(over)
    c = cache(**over.pop("cache", {}))
    size = abi.m2_attn_tree_kv4_workspace_bytes(32, 8, 128)
    base = dict(q=FAKE, ld_q=4096, out=FAKE, ld_o=4096, H=32, cu_nodes=[0, 3, 8], parent=FAKE, kv_pos=FAKE, scale=0.1,
                ws=FAKE, ws_bytes=size)
    if over.get("ws_bytes") == -1:
        over["ws_bytes"] = size - 1
    refused(abi.m2_attn_tree_kv4, base, over, want, c)


def test_offsets_have_to_match_the_cache():
    for call in (lambda: abi.m2_kv4_keep(cache(), [0, 3], FAKE, FAKE, FAKE),
                 lambda: abi.m2_attn_tree_kv4(cache(), FAKE, 4096, FAKE, 4096, 32, [0, 3], FAKE, FAKE, 0.1, FAKE, 1 << 40)):
        with pytest.raises(abi.M2Error):
            call()


def _layer():
    return abi.M2Layer(FAKE, abi.M2Weight(FAKE, FAKE, 18560, 4096, abi.M2_W_FP8_BLOCK128), FAKE, FAKE, FAKE, FAKE, FAKE,
                       FAKE, abi.M2Weight(FAKE, FAKE, 4096, 8192, abi.M2_W_FP8_BLOCK128))


@pytest.mark.parametrize("over,want", TREES + [
    (dict(hidden=None), A), (dict(hidden=FAKE + 2), L), (dict(parent=None), A), (dict(parent=FAKE + 2), L),
    (dict(ssm_state=None), A), (dict(ssm_state=FAKE + 8), L), (dict(conv_state=FAKE + 4), L), (dict(conv_pos=None), A),
    (dict(ws=None), W), (dict(ws=FAKE + 128), W), (dict(ws_bytes=-1), W)])
def test_layer_refuses(over, want):
    d = abi.dims_struct(synth.NEMOTRON_H_8B)
    size = abi.m2_workspace_bytes_tree(d, 2, 8)
    base = dict(hidden=FAKE, cu_nodes=[0, 3, 8], parent=FAKE, ssm_state=FAKE, conv_state=FAKE, conv_pos=FAKE, ws=FAKE,
                ws_bytes=size)
    over = dict(over)
    if over.get("ws_bytes") == -1:
        over["ws_bytes"] = size - 1
    refused(abi.mamba2_layer_tree, base, over, want, d, _layer())
    if "hidden" not in over and "parent" not in over:
        base = {k: v for k, v in base.items() if k not in ("hidden", "parent")} | dict(path=FAKE, count=FAKE)
        refused(abi.mamba2_layer_tree_commit, base, over, want, d, _layer())
    for gone in ("path", "count"):
        base = dict(cu_nodes=[0, 3, 8], path=FAKE, count=FAKE, ssm_state=FAKE, conv_state=FAKE, conv_pos=FAKE, ws=FAKE,
                    ws_bytes=size)
        refused(abi.mamba2_layer_tree_commit, base, {gone: None}, A, d, _layer())


def test_workspace_sizes():
    d = abi.dims_struct(synth.NEMOTRON_H_8B)
    assert 0 < abi.m2_workspace_bytes_tree(d, 1, 5) < abi.m2_workspace_bytes_tree(d, 16, 256)
    assert abi.m2_workspace_bytes_tree(d, 0, 5) == 0
    assert abi.m2_attn_tree_kv4_workspace_bytes(30, 8, 128) == 0 and abi.m2_attn_tree_kv4_workspace_bytes(32, 8, 96) == 0
    m = abi.m2_workspace_map(d, abi.M2_WS_KIND_TREE, 2, [0, 3, 8])
    assert {"xn", "zx", "u", "y", "g", "unscale"} == set(m) and max(m.values()) < abi.m2_workspace_bytes_tree(d, 2, 8)


def test_reference_paths():
    assert ref.paths([-1, 0, 0, 2, -1, 4, 7, 5, -2, 8]) == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [4, 5], [], [4, 5, 7], [], []]


def test_reference_scan_is_the_steps_of_each_path():
    rng, g = random.Random(1), torch.Generator().manual_seed(1)
    H, P, N, G, n = 4, 3, 5, 2, 9
    r = lambda *s: torch.randn(*s, generator=g, dtype=ref.F)  # noqa: E731
    h, x, B, C, dt, b, al, D = r(H, P, N), r(n, H, P), r(n, G, N), r(n, G, N), r(n, H), r(H), r(H).abs(), r(H)
    parent = ref.random_parents(n, rng, "forest")
    y, size = ref.ssm(h, x, B, C, dt, b, al, D, parent)
    step, keep = ref.steps(dt, b, al)
    for k, path in enumerate(ref.paths(parent)):  # the closed form of the header
        s = lambda a: sum(torch.log(keep[i]) for i in path[:path.index(a) + 1])  # noqa: E731
        group = torch.arange(H) // (H // G)
        want = torch.exp(s(k))[:, None] * torch.einsum("hn,hpn->hp", C[k][group], h) + D[:, None] * x[k]
        for j in path:
            cb = (C[k] * B[j]).sum(-1)[group]
            want = want + (torch.exp(s(k) - s(j)) * step[j] * cb)[:, None] * x[j]
        assert torch.allclose(y[k], want, rtol=1e-12, atol=1e-12) and bool((size[k] >= y[k].abs() - 1e-9).all())


def test_reference_verification_keeps_the_target_distribution():
    """Two siblings drawn from q, then the draw: the first token after the root is distributed as p."""
    g = torch.Generator().manual_seed(3)
    V, N = 5, 40000
    p = torch.softmax(torch.randn(3, V, generator=g, dtype=ref.F), -1)
    q = torch.softmax(torch.randn(3, V, generator=g, dtype=ref.F), -1)
    tok = torch.multinomial(q[0], 2 * N, replacement=True, generator=g).tolist()
    u = torch.rand(N, 4, generator=g, dtype=ref.F).tolist()
    hits = torch.zeros(V, dtype=ref.F)
    for i in range(N):
        token = [0, tok[2 * i], tok[2 * i + 1]]
        path, last = ref.verify(p, q, [-1, 0, 0], token, [0, u[i][0], u[i][1]], u[i][2])
        hits[token[path[1]] if len(path) > 1 else last] += 1
    # binomial spread: five standard deviations
    assert bool(((hits / N - p[0]).abs() < 5 * (p[0] * (1 - p[0]) / N).sqrt()).all())


# ------------------------------------------------------------------ holders (on the CPU: no kernel is launched)

class Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("w8a16_gemv", "m2_qk_norm_rope", "m2_kv4_append", "m2_attn_tree_kv4", "m2_kv4_keep", "mamba2_layer_tree",
                 "mamba2_layer_tree_commit"):
        monkeypatch.setattr(abi, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    return seen


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_attention_holder_checks_its_trees(calls):
    from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache
    m = DeviceAttention(synth.make_attention(synth.TINY_ATTENTION, 9), device="cpu")
    cache = Kv4Cache(2, 2, 12, 256, m.Hkv, m.D, device="cpu")
    bf = torch.bfloat16
    good = dict(x=torch.zeros(5, m.hidden, dtype=bf), cu=[0, 3, 5], parent=ints(-1, 0, 0, -1, 0), row_pos=ints(0, 1, 1, 0, 1),
                b=m.buffers(8, 0, 2, trees=True), out=torch.zeros(5, m.hidden, dtype=bf))

    def tree(**over):
        a = dict(good, **over)
        m.tree(a["x"], a["cu"], a["parent"], a["row_pos"], cache, 1, a["b"], a["out"], Stream())
    tree()
    assert [n for n, _ in calls] == ["w8a16_gemv", "m2_qk_norm_rope", "m2_kv4_append", "m2_attn_tree_kv4", "w8a16_gemv"]
    for over in (dict(cu=[0, 5]), dict(parent=ints(-1, 0, 0, -1)), dict(parent=torch.zeros(5, dtype=torch.int64)),
                 dict(x=torch.zeros(4, m.hidden, dtype=bf)), dict(out=torch.zeros(6, m.hidden, dtype=bf)),
                 dict(row_pos=ints(0, 1, 1, 0)), dict(b=m.buffers(4, 0, 2, trees=True)), dict(b=m.buffers(8, 0, 2)),
                 dict(parent=torch.zeros(10, dtype=torch.int32)[::2])):
        with pytest.raises(abi.M2Error):
            tree(**over)
    assert len(calls) == 5
    path, count = ints(0, 2, -1, 0, -1), ints(2, 1)
    with pytest.raises(abi.M2Error):
        cache.keep([0, 5], path, count, 0)
    with pytest.raises(abi.M2Error):
        cache.keep([0, 3, 5], path, ints(2), 0)
    with pytest.raises(abi.M2Error):
        cache.keep([0, 3, 5], ints(0, 2), count, 0)
    assert len(calls) == 5


def test_layer_holder_checks_its_trees(calls):
    from mamba_ssm_layer_gb300.layer import DeviceLayer
    dl = DeviceLayer(synth.make_layer(synth.TINY, synth.WL_TINY_DECODE), device="cpu")
    st, ws = dl.new_state(2, device="cpu"), dl.workspace_tree(2, 5, device="cpu")
    x = torch.zeros(5, 256, dtype=torch.int16)
    dl.tree(x, [0, 3, 5], ints(-1, 0, 0, -1, 0), st, ws, Stream())
    dl.tree_commit([0, 3, 5], ints(0, 1, -1, 0, -1), ints(2, 1), st, ws, Stream())
    assert [n for n, _ in calls] == ["mamba2_layer_tree", "mamba2_layer_tree_commit"]
    for bad in (lambda: dl.tree(x, [0, 5], ints(-1, 0, 0, -1, 0), st, ws, Stream()),
                lambda: dl.tree(x[:4], [0, 3, 5], ints(-1, 0, 0, -1, 0), st, ws, Stream()),
                lambda: dl.tree(x.float(), [0, 3, 5], ints(-1, 0, 0, -1, 0), st, ws, Stream()),
                lambda: dl.tree(x, [0, 3, 5], ints(-1, 0, 0), st, ws, Stream()),
                lambda: dl.tree_commit([0, 3, 5], ints(0, 1), ints(2, 1), st, ws, Stream()),
                lambda: dl.tree_commit([0, 3, 5], ints(0, 1, -1, 0, -1), ints(2), st, ws, Stream())):
        with pytest.raises(abi.M2Error):
            bad()
    assert len(calls) == 2
