"""Calls of the operators for trees of drafted tokens that their documentation allows and
ordinary use seldom makes.  Tolerances as in test_gpu_tree.py."""
import random

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from mamba_ssm_layer_gb300.layer import _empty
from tests import attention_ref
from tests import tree_ref as ref
from tests.test_gpu_attention import BF16, EVAL, F16, Cache, close, gen, offsets, out_rows, rows
from tests.test_gpu_tree import Ssm, ints, paths_of, run_tree, trees

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


# ------------------------------------------------------------------ sizes that change how work is dealt out

@pytest.mark.parametrize("C,K,lens", [(64, 4, [64, 0, 3] * 20), (2048, 2, [1, 5, 64, 63, 62, 2] * 12), (1032, 8, [64] * 14),
                                      (37, 4, [9, 64, 1] * 24), (8, 3, [5] * 300)])
def test_conv_of_many_nodes(C, K, lens):
    """Several nodes a block, pieces that end with their sequence, and more sequences than one launch takes."""
    g, cu, T = gen(C), offsets(lens), sum(lens)
    parents = trees(lens, "tree", C)
    for i in range(0, len(lens), 7):
        if lens[i] > 2:
            parents[i][lens[i] // 2] = -5  # a padded place
    x, ring = rows(T, C, g, 8), rows(len(lens) * (K - 1), C, g).view(len(lens), K - 1, C)
    w, b = rows(C, K, g, spread=0.5), rows(1, C, g)[0]
    pos = list(range(len(lens)))
    buf, out = out_rows(T, C, 8)
    abi.mamba2_tree_conv(ring, ints(pos), x, x.stride(0), w, b, out, out.stride(0), cu, ints([p for t in parents for p in t]),
                         C, K)
    assert bool((buf[:, :8] == 7).all())
    for i, t in list(enumerate(parents))[::5]:
        want, size = ref.conv(ring[i], pos[i], x[cu[i]:cu[i + 1]], w, b, t, 1)
        close(out[cu[i]:cu[i + 1]], want, BF16 * want.abs() + 2.0 ** -19 * size + 1e-38)
    # and every node is the one that a call for its sequence alone gives
    for i, t in enumerate(parents):
        if t:
            one = _empty((len(t), C), bf, "cuda")
            abi.mamba2_tree_conv(ring[i], ints(pos[i:i + 1]), x[cu[i]:], x.stride(0), w, b, one, C, [0, len(t)], ints(t), C, K)
            assert torch.equal(one, out[cu[i]:cu[i + 1]]), i


@pytest.mark.parametrize("H,P,N,G", [(48, 16, 16, 2), (21, 8, 32, 1), (64, 72, 16, 4), (40, 20, 128, 2)])
@pytest.mark.parametrize("lens", [[7], [16, 0, 2] * 7, [5] * 100, [1] * 300, [33, 2] * 30, [17] * 20])
def test_ssm_whatever_the_heads_of_a_block(H, P, N, G, lens):
    parents, cu = trees(lens, "tree", H), offsets(lens)
    s = Ssm(len(lens), sum(lens), H, P, N, G, N + P, extra=4)
    y = s.run(cu, parents)
    pick = sorted({0, len(lens) - 1, len(lens) // 2, min(128, len(lens) - 1)})
    kept = [t if i in pick else [] for i, t in enumerate(parents)]
    s.check(y, cu, kept)


def test_commit_and_keep_of_many_sequences():
    B, H, P, N, G, K, D, Hkv = 300, 4, 8, 16, 2, 4, 64, 2
    rng = random.Random(1)
    lens = [rng.choice([0, 1, 4, 9]) for _ in range(B)]
    parents, cu, T = trees(lens, "tree", 2), offsets(lens), sum(lens)
    picked, flat = paths_of(parents, rng)
    s = Ssm(B, T, H, P, N, G, 4, extra=4)
    W = s.W
    ring, pos = rows(B * (K - 1), W, gen(2)).view(B, K - 1, W), ints([rng.randrange(1000) for _ in range(B)])
    count = ints([len(p) for p in picked])
    out = torch.empty_like(s.h), torch.empty_like(ring), torch.empty_like(pos)
    abi.mamba2_tree_commit(s.h, ring, pos, *out, s.u, s.u.stride(0), s.u, s.u.stride(0), s.dt, s.dt.stride(0), s.A_log,
                           s.dt_bias, cu, ints(flat), count, H, P, N, G, K)
    for i, path in enumerate(picked):  # alone
        one = s.h[i:i + 1].clone(), ring[i:i + 1].clone(), pos[i:i + 1].clone()
        if path:
            at = slice(cu[i], cu[i + 1])
            abi.mamba2_tree_commit(one[0], one[1], one[2], *one, s.u[at], s.u.stride(0), s.u[at], s.u.stride(0), s.dt[at],
                                   s.dt.stride(0), s.A_log, s.dt_bias, [0, lens[i]], ints(flat[at]), count[i:i + 1].clone(),
                                   H, P, N, G, K)
        assert torch.equal(out[0][i], one[0][0]) and torch.equal(out[1][i], one[1][0]) and int(out[2][i]) == int(one[2]), i
    pasts = [rng.randrange(130) for _ in range(B)]
    c = Cache([a + b for a, b in zip(lens, pasts)], Hkv, D, 3)
    ce = offsets([a + b for a, b in zip(lens, pasts)])
    k0, v0 = c.gather(ce)
    abi.m2_kv4_keep(c.struct, cu, ints(flat), count, ints(pasts))
    k1, v1 = c.gather(ce)
    for i, path in enumerate(picked):
        src = list(range(pasts[i] + lens[i]))
        for j, r in enumerate(path):
            src[pasts[i] + j] = pasts[i] + r
        src = torch.tensor(src, dtype=torch.long, device="cuda") + ce[i]
        assert torch.equal(k1[ce[i]:ce[i + 1]].view(torch.int16), k0[src].view(torch.int16))
        assert torch.equal(v1[ce[i]:ce[i + 1]].view(torch.int16), v0[src].view(torch.int16))


def test_keep_of_a_path_that_names_a_node_twice():
    """As if all rows were read before any is written: nodes in any order, one of them twice."""
    c = Cache([80], 2, 64, 1)
    k0, v0 = c.gather([0, 80])
    path = [5, 0, 9, 5, 1]
    abi.m2_kv4_keep(c.struct, [0, 20], ints(path + [-1] * 15), ints([5]), ints([60]))
    k1, v1 = c.gather([0, 80])
    src = list(range(80))
    src[60:65] = [60 + r for r in path]
    assert torch.equal(k1.view(torch.int16), k0[src].view(torch.int16))
    assert torch.equal(v1.view(torch.int16), v0[src].view(torch.int16))


@pytest.mark.parametrize("H,lens", [(32, [3, 4]), (32, [5, 9]), (32, [64, 40])])
def test_attention_over_pages_far_into_a_large_pool(H, lens):
    """Pages whose bytes lie past 2^32 of the pool's start."""
    Hkv, D, first = 8, 128, 60000  # 60000 pages of 73728 bytes
    pasts = [300, 64]
    ends = [a + b for a, b in zip(lens, pasts)]
    parents, cu, ce = trees(lens, "tree", 1), offsets(lens), offsets(ends)
    g = gen(7)
    q, k, v = rows(cu[-1], H * D, g), rows(ce[-1], Hkv * D, g), rows(ce[-1], Hkv * D, g)
    outs = []
    for where in (first, 0):
        c = Cache(ends, Hkv, D, 5, first_page=where)
        c.append(k, v, ce, [0, 0])
        ws = _empty((abi.m2_attn_tree_kv4_workspace_bytes(H, Hkv, D),), torch.uint8, "cuda")
        out = _empty((cu[-1], H * D), bf, "cuda")
        abi.m2_attn_tree_kv4(c.struct, q, H * D, out, H * D, H, cu, ints([p for t in parents for p in t]), ints(pasts),
                             D ** -0.5, ws, ws.numel())
        picked = [ref.paths(t)[-1] for t in parents]
        flat = [x for p, t in zip(picked, parents) for x in p + [-1] * (len(t) - len(p))]
        abi.m2_kv4_keep(c.struct, cu, ints(flat), ints([len(p) for p in picked]), ints(pasts))
        kept = c.gather(ce)
        outs.append((out, *kept))
        if where:
            assert c.pages.numel() > 2 ** 32 and int(c.table.max()) * Hkv * 72 * D > 2 ** 32
        del c
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    kk, vv = (attention_ref.rounded_rows(t.reshape(-1, Hkv, D)) for t in (k, v))
    for i, t in enumerate(parents):
        r, e = slice(cu[i], cu[i + 1]), slice(ce[i], ce[i + 1])
        want, size, total, score = ref.attend(q[r].reshape(-1, H, D), kk[e], vv[e], D ** -0.5, pasts[i], t)
        close(outs[0][0][r].reshape(-1, H, D), want,
              BF16 * want.abs() + (F16 + EVAL + 2.0 ** -19 * score) * size + 2.0 ** -32 * total + 1e-30)


@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 128), (8, 2, 64), (16, 1, 64)])
@pytest.mark.parametrize("n", [1, 4, 5, 16, 17, 33])
def test_attention_of_short_and_long_together(H, Hkv, D, n):
    """Runs and spans that end within a page, a tile's start, or a tile; as many sequences as a launch takes and more."""
    rng = random.Random(n)
    lens = [rng.choice([0, 1, n, n]) for _ in range(140)]
    pasts = [rng.choice([0, 1, 31, 32, 33, 63, 64, 65, 500]) for _ in lens]
    lens[0], pasts[0] = n, 1500
    run_tree(lens, pasts, H, Hkv, D, seed=n)


@pytest.mark.parametrize("H,Hkv,D,n", [(4, 4, 128, 8), (4, 2, 128, 4), (32, 8, 128, 2), (8, 8, 64, 7), (6, 2, 64, 2), (8, 1, 64, 1),
                                       (3, 3, 128, 5), (16, 16, 64, 8)])
def test_attention_of_few_rows(H, Hkv, D, n):
    """At most 8 rows a kv head, at every kind of length and cut."""
    rng = random.Random(H + n)
    for seed, pasts in enumerate(([0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 500], [3000], [700, 0, 40, 9] * 35)):
        lens = [n if i % 3 < 2 else rng.randrange(n + 1) for i in range(len(pasts))]
        run_tree(lens, pasts, H, Hkv, D, seed=seed)
    run_tree([n, n], [20, 9000], H, Hkv, D, kind="chain", spread=30.0, seed=5, width=400)


# ------------------------------------------------------------------ waits, streams, graphs

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [5, 64])
def test_attention_times_out_cleanly(D, n):
    """Waits that give up at once: the status says so, and the same call computes correctly afterwards."""
    c, q, want, (cu, parents, pasts, ws, scale) = run_tree([n, n - 1], [700, 3000], 32, 8, D)
    flat = ints([p for t in parents for p in t])

    def run():
        out = torch.empty_like(want)
        abi.m2_attn_tree_kv4(c.struct, q, q.stride(0), out, out.stride(0), 32, cu, flat, ints(pasts), scale, ws, ws.numel())
        return out, abi.m2_device_status(clear=True)
    first = run()
    assert first[1] == abi.M2_OK and torch.equal(first[0], want)
    try:
        abi.m2_set_wait_limit(1)
        assert run()[1] == abi.M2_ERR_TIMEOUT
        abi.m2_set_wait_limit(900000)
        again = run()
        assert again[1] == abi.M2_OK and torch.equal(again[0], want)
    finally:
        abi.m2_set_wait_limit(0)
    again = run()
    assert again[1] == abi.M2_OK and torch.equal(again[0], want)


class Step:
    """All operators in the order in which a step uses them, on one stream, from what `fill` puts in place."""

    def __init__(self, lens=(5, 0, 20), past=(70, 3, 200), H=16, Hkv=4, D=64, V=500):
        self.lens, self.H, self.Hkv, self.D, self.V = list(lens), H, Hkv, D, V
        self.cu, T, B = offsets(lens), sum(lens), len(lens)
        self.s = Ssm(B, T, 4, 16, 32, 2, 3, extra=4)
        W, self.K = self.s.W, 4
        self.cache = Cache([a + b + 70 for a, b in zip(past, lens)], Hkv, D, 2)
        ce = offsets([a + 70 for a in past])  # a context of real values
        self.cache.append(rows(ce[-1], Hkv * D, gen(10)), rows(ce[-1], Hkv * D, gen(11)), ce, [0] * B)
        self.kv = rows(T, 2 * Hkv * D, gen(1))
        self.q, self.out = rows(T, H * D, gen(2)), _empty((T, H * D), bf, "cuda")
        self.xbc, self.u = rows(T, W, gen(3)), _empty((T, W), bf, "cuda")
        self.w, self.b = rows(W, self.K, gen(4), spread=0.5), rows(1, W, gen(5))[0]
        self.ring, self.pos = rows(B * 3, W, gen(6)).view(B, 3, W), ints([3, 4, 5])
        self.y = _empty((T, 64), torch.float32, "cuda")
        self.p, self.qd = (torch.softmax(2 * torch.randn(T, V, device="cuda", generator=gen(k)), -1) for k in (8, 8))
        self.rand, self.rand_next = (torch.rand(n, device="cuda", generator=gen(9)) for n in (T, B))
        self.past, self.parent, self.token = ints(list(past)), ints([0] * T), ints([0] * T)
        self.path, self.count, self.next = ints([0] * T), ints([0] * B), ints([0] * B)
        self.ws = _empty((abi.m2_attn_tree_kv4_workspace_bytes(H, Hkv, D),), torch.uint8, "cuda")
        self.state = [self.s.h, self.ring, self.pos, self.cache.pages]
        self.start = [t.clone() for t in self.state]

    def source(self, seed):
        g, T = gen(seed), self.cu[-1]
        parents = trees(self.lens, "tree", seed)
        return [torch.tensor([x for t in parents for x in t], dtype=torch.int32, device="cuda"),
                torch.randint(0, self.V, (T,), device="cuda", generator=g, dtype=torch.int32),
                rows(T, self.q.shape[1], g), rows(T, self.xbc.shape[1], g), torch.rand(T, device="cuda", generator=g)]

    def fill(self, source):
        for d, x in zip([self.parent, self.token, self.q, self.xbc, self.rand], source):
            d.copy_(x)
        for d, x in zip(self.state, self.start):
            d.copy_(x)

    def run(self, stream):
        s, c, W, KD = self.s, self.cache.struct, self.s.W, self.Hkv * self.D
        abi.mamba2_tree_conv(self.ring, self.pos, self.xbc, W, self.w, self.b, self.u, W, self.cu, self.parent, W, self.K, 1,
                             stream)
        abi.mamba2_tree_ssm(s.h, self.u, self.u[:, 64:], self.u[:, 128:], W, s.dt, s.dt.stride(0), s.A_log, s.D, s.dt_bias,
                            self.y, self.cu, self.parent, 4, 16, 32, 2, stream)
        abi.m2_kv4_append(c, self.kv, 2 * KD, self.kv[:, KD:], 2 * KD, self.cu, self.past, stream)
        abi.m2_attn_tree_kv4(c, self.q, self.H * self.D, self.out, self.H * self.D, self.H, self.cu, self.parent, self.past,
                             0.125, self.ws, self.ws.numel(), stream)
        abi.m2_verify_tree(self.p, self.V, self.qd, self.V, abi.M2_PROB_F32, self.V, self.cu, self.parent, self.token, self.rand,
                           self.rand_next, self.path, self.count, self.next, stream)
        abi.mamba2_tree_commit(s.h, self.ring, self.pos, s.h, self.ring, self.pos, self.xbc, W, self.u, W, s.dt, s.dt.stride(0),
                               s.A_log, s.dt_bias, self.cu, self.path, self.count, 4, 16, 32, 2, self.K, stream)
        abi.m2_kv4_keep(c, self.cu, self.path, self.count, self.past, stream)

    def results(self):
        return [t.clone() for t in (self.u, self.y, self.out, self.path, self.count, self.next, *self.state)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


LENS = [(5, 0, 20), (4, 0, 3), (64, 0, 9)]


@pytest.mark.parametrize("lens", LENS)
def test_operators_run_on_their_stream(lens):
    """Inputs that a side stream makes behind a long kernel, with no other order than the stream's own."""
    st = Step(lens)
    a, b = st.source(1), st.source(2)
    st.fill(a)
    st.run(torch.cuda.current_stream())
    want = st.results()
    st.fill(b)
    st.run(torch.cuda.current_stream())
    assert not same(st.results(), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        st.fill(a)
    st.run(side)
    with torch.cuda.stream(side):
        got = st.results()
    side.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("lens", LENS)
def test_graphs_of_one_workspace_and_other_trees(lens):
    """Two captured steps share every buffer; what is replayed has other trees, paths and tokens than what was captured."""
    st = Step(lens)
    side = torch.cuda.Stream()
    st.fill(st.source(0))
    st.run(torch.cuda.current_stream())  # (attributes of kernels are set outside of a capture)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            st.run(side)
        graphs.append(g)
    for seed in (3, 4, 5):
        st.fill(st.source(seed))
        st.run(torch.cuda.current_stream())
        want = st.results()
        for g in graphs:
            st.fill(st.source(seed))
            g.replay()
            assert same(st.results(), want)


@pytest.mark.parametrize("lens", LENS)
def test_two_calls_at_once(lens):
    """Two streams, their own buffers and workspaces each."""
    a, b = Step(lens), Step((2, 0, 16))
    sa, sb = a.source(6), b.source(7)
    want = []
    for st, src in ((a, sa), (b, sb)):
        st.fill(src)
        st.run(torch.cuda.current_stream())
        want.append(st.results())
        st.fill(src)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, src, s in ((a, sa, streams[0]), (b, sb, streams[1])):
            with torch.cuda.stream(s):
                st.fill(src)
            st.run(s)
    torch.cuda.synchronize()
    assert same(a.results(), want[0]) and same(b.results(), want[1])
