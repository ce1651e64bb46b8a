"""The operators for trees of drafted tokens against their 64-bit plain forms.

Tolerances count roundings: bf16 2^-8 of the value, f16 2^-11.  Sums in fp32 are off by at
most 2^-24 of the sum of |terms| an addition; the matrix instructions cut rather than
round (2^-23) and add 16 terms at a time.
  conv   up to 9 additions and the activation (a few 2^-23): 2^-19 of the sum of |terms|
  ssm    at most 24 + 12 accumulations of 2^-23 and as much again within them: 2^-17; a
         log decay is off by 2^-21 of itself (exp, log1p, product), so a path's factor by
         |s| 2^-21
  attention as in test_gpu_attention.py, and for far ranges: a score's 8 accumulations cut 2^-23
         of its sum of |terms| each, which is 2^-20 of it in a probability, and as much again
         in their sum; a probability below f16's normal range is off by half a step, 2^-25, in
         units of 2^-7 of the row's largest, so that the output is off by 2^-32 of sum |v|"""
import random

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from mamba_ssm_layer_gb300.layer import _empty
from tests import attention_ref
from tests import tree_ref as ref
from tests.test_gpu_attention import BF16, EVAL, F16, Cache, close, gen, offsets, out_rows, rows

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


def ints(v):
    t = _empty((max(len(v), 1),), torch.int32, "cuda")
    t[:len(v)].copy_(torch.tensor(v, dtype=torch.int32))
    return t


def trees(lens, kind, seed=0):
    rng = random.Random(seed)
    return [ref.random_parents(n, rng, kind) if n else [] for n in lens]


def paths_of(parents, rng):
    """An accepted path a tree (of any node), and the flat array of the entry points."""
    picked = [ref.paths(p)[rng.randrange(len(p))] if p else [] for p in parents]
    flat = [x for p, t in zip(picked, parents) for x in p + [-1] * (len(t) - len(p))]
    return picked, flat


# ------------------------------------------------------------------ conv

@pytest.mark.parametrize("C,K,extra,silu,bias", [(640, 4, 16, 1, True), (64, 2, 0, 0, True), (1032, 8, 8, 1, False),
                                                 (37, 4, 3, 1, True), (6, 3, 0, 0, False), (2048, 5, 0, 1, True)])
@pytest.mark.parametrize("kind", ["chain", "star", "tree", "forest", "padded"])
def test_conv(C, K, extra, silu, bias, kind):
    g, lens = gen(C + K), [1, 0, 7, 64, 33]
    cu, T = offsets(lens), sum(lens)
    parents = trees(lens, "tree" if kind == "padded" else kind, C)
    if kind == "padded":  # places without a node, and nodes below them
        parents[2][3], parents[3][40], parents[4] = -2, 40, [-1] + list(range(16)) + [-7] * 16
        parents[3][50] = 40
    x = rows(T, C, g, extra)
    ring = rows(len(lens) * (K - 1), C, g).view(len(lens), K - 1, C)
    w, b = rows(C, K, g, spread=0.5), rows(1, C, g)[0] if bias else None
    pos = [0, 3, 1000003, 5, 2 ** 31 - 70]
    buf, out = out_rows(T, C, extra)
    abi.mamba2_tree_conv(ring, ints(pos), x, x.stride(0), w, b, out, out.stride(0), cu,
                         ints([p for t in parents for p in t]), C, K, silu)
    for i, t in enumerate(parents):
        want, size = ref.conv(ring[i], pos[i], x[cu[i]:cu[i + 1]], w, b, t, silu)
        close(out[cu[i]:cu[i + 1]], want, BF16 * want.abs() + 2.0 ** -19 * size + 1e-38)
    assert bool((buf[:, :extra] == 7).all())


@pytest.mark.parametrize("C,K", [(256, 4), (41, 3)])
def test_conv_of_a_chain_is_the_single_token_conv(C, K):
    g, n, B = gen(5), 9, 3
    x = rows(B * n, C, g).view(B, n, C)
    ring, w, b = rows(B * (K - 1), C, g).view(B, K - 1, C), rows(C, K, g), rows(1, C, g)[0]
    pos = ints([4, 0, 77])
    out = _empty((B, n, C), bf, "cuda")
    abi.mamba2_tree_conv(ring, pos, x, C, w, b, out, C, offsets([n] * B), ints(list(range(-1, n - 1)) * B), C, K)
    one = _empty((B, C), bf, "cuda")
    for j in range(n):
        abi.conv1d_update(ring, pos, x[:, j].contiguous(), C, w, b, one, B, C, K, 1)
        assert torch.equal(one, out[:, j])


# ------------------------------------------------------------------ SSM outputs

class Ssm:
    def __init__(self, nseq, T, H, P, N, G, seed, extra=0, spread=1.0, far=1.0):
        g = gen(seed)
        self.H, self.P, self.N, self.G, self.T = H, P, N, G, T
        self.W = H * P + 2 * G * N
        self.h = _empty((nseq, H, P, N), torch.float32, "cuda")
        self.h.copy_(torch.randn(nseq, H, P, N, device="cuda", generator=g) * spread)
        self.u = rows(T, self.W, g, extra)
        self.dt = rows(T, H, g, 5, far)
        f = lambda t: _empty(t.shape, torch.float32, "cuda").copy_(t)  # noqa: E731
        self.A_log, self.D = f(torch.rand(H, device="cuda", generator=g) * 2.7), f(1 + 0.1 * torch.randn(H, device="cuda", generator=g))
        self.dt_bias = f(torch.randn(H, device="cuda", generator=g) - 3)

    def parts(self, u=None):
        u = self.u if u is None else u
        T, H, P, N, G = len(u), self.H, self.P, self.N, self.G
        return (u[:, :H * P].reshape(T, H, P), u[:, H * P:H * P + G * N].reshape(T, G, N),
                u[:, H * P + G * N:].reshape(T, G, N))

    def run(self, cu, parents, stream=None):
        H, P, N, G, u = self.H, self.P, self.N, self.G, self.u
        y = _empty((self.T, H * P), torch.float32, "cuda")
        y.fill_(7.0)
        before = self.h.clone()
        abi.mamba2_tree_ssm(self.h, u, u[:, H * P:], u[:, H * P + G * N:], u.stride(0), self.dt, self.dt.stride(0),
                            self.A_log, self.D, self.dt_bias, y, cu, ints([p for t in parents for p in t]), H, P, N, G,
                            stream)
        assert torch.equal(self.h, before)
        return y

    def check(self, y, cu, parents, bad=None):
        x, B, C = self.parts()
        for i, t in enumerate(parents):
            r = slice(cu[i], cu[i + 1])
            if not t:
                continue
            want, size = ref.ssm(self.h[i], x[r], B[r], C[r], self.dt[r], self.dt_bias, self.A_log, self.D, t)
            s = ref.ancestors_sum(t, torch.log(ref.steps(self.dt[r], self.dt_bias, self.A_log)[1])).abs()[..., None]
            close(y[r].view(-1, self.H, self.P), want, (2.0 ** -17 + s * 2.0 ** -21) * size + 1e-30)


@pytest.mark.parametrize("H,P,N,G", [(8, 64, 128, 2), (8, 32, 16, 1), (6, 24, 32, 3), (3, 20, 64, 1), (4, 7, 128, 2),
                                     (2, 256, 64, 2), (4, 1, 16, 4), (40, 64, 128, 1)])
@pytest.mark.parametrize("lens,kind", [([1], "chain"), ([5, 0, 16], "tree"), ([17, 32, 1], "forest"), ([64, 33], "tree"),
                                       ([64], "chain"), ([64], "star")])
def test_ssm(H, P, N, G, lens, kind):
    parents, cu = trees(lens, kind, H), offsets(lens)
    s = Ssm(len(lens), sum(lens), H, P, N, G, N + P, extra=8 if P % 2 else 4)
    s.check(s.run(cu, parents), cu, parents)


def test_ssm_of_long_decays_and_padded_places():
    parents = [list(range(-1, 63)), [-1, 0, 5, 1, -9, 3, 2, 0] + [-2] * 20]
    lens = [len(t) for t in parents]
    s = Ssm(2, sum(lens), 4, 32, 64, 2, 3, far=2.0)
    s.dt_bias.add_(3.0)  # factors down to e^-100 and beyond over a path
    s.u[lens[0] + 8:].fill_(float("nan"))  # what no node holds
    s.dt[lens[0] + 8:].fill_(float("nan"))
    y = s.run(offsets(lens), parents)
    s.check(y, offsets(lens), parents)
    for r in (2, 4, 6, *range(8, 28)):
        assert bool((y[lens[0] + r] == 0).all())


@pytest.mark.parametrize("P", [64, 9])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_ssm_bad_values_reach_only_the_nodes_below(P, what, value):
    parents = [[-1, 0, 0, 1, 2, 3, 1, 6, 4, 4, 0, 10, 11, 12, 0, 14, 15, 16, 2, 18]]
    n, at = len(parents[0]), 6
    s = Ssm(1, n, 4, P, 32, 2, 8)
    good = s.run([0, n], parents)
    x, B, C = (slice(0, 4 * P), slice(4 * P, 4 * P + 64), slice(4 * P + 64, 4 * P + 128))
    if what == "dt":
        s.dt[at, 1] = value
    else:
        s.u[at, dict(x=x, B=B, C=C)[what].start + 3] = value
    y = s.run([0, n], parents)
    hit = {"C": [at]}.get(what, [r for r, p in enumerate(ref.paths(parents[0])) if at in p])
    other = [r for r in range(n) if r not in hit]
    assert torch.equal(y[other], good[other])
    if what == "dt":  # the step's clamp takes NaN to its lower end, infinity to its upper one (mamba2_ssm_step does)
        s.dt[at, 1] = 1e30 if value == float("inf") else -200.0
        assert torch.equal(y, s.run([0, n], parents))
        return
    for r in hit:
        assert not bool(y[r].isfinite().all()), r
        if what == "x" and r == at:
            assert int((~y[r].isfinite()).sum()) == 1  # one channel
    if what == "x" and value == float("inf"):
        assert bool(y[at, 3].isinf())


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("H,P,N,G,K", [(8, 64, 128, 2, 4), (6, 24, 32, 3, 2), (3, 20, 64, 1, 8), (4, 7, 16, 2, 3)])
@pytest.mark.parametrize("place", ["in place", "apart"])
def test_commit_is_the_steps_of_the_path(H, P, N, G, K, place):
    lens = [5, 0, 64, 1, 17]
    parents, cu, B = trees(lens, "tree", K), offsets([5, 0, 64, 1, 17]), 5
    s = Ssm(B, sum(lens), H, P, N, G, 4, extra=4)
    g = gen(K)
    W, T = s.W, sum(lens)
    xbc = rows(T, W, g, 8)
    ring = rows(B * (K - 1), W, g).view(B, K - 1, W)
    pos = ints([0, 9, 70001, 2, 3])
    picked, flat = paths_of(parents, random.Random(K))
    picked[4], flat[cu[4]:] = [], [-1] * 17  # nothing kept
    count = ints([len(p) for p in picked])
    # the same as single tokens
    h1, ring1, pos1 = s.h.clone(), ring.clone(), pos.clone()
    for i, path in enumerate(picked):
        for r in path:
            t = cu[i] + r
            u = s.u[t:t + 1].contiguous()
            u = torch.cat([u, u.new_zeros(1, -W % 4)], 1)
            y = torch.empty(1, H * P, device="cuda")
            dt = s.dt[t:t + 1].contiguous()
            abi.mamba2_ssm_step(h1[i:i + 1], u, u[:, H * P:], u[:, H * P + G * N:], dt, u.shape[1], s.A_log, s.D, s.dt_bias, y,
                                1, H, P, N, G)
            ring1[i, int(pos1[i]) % (K - 1)] = xbc[t]
            pos1[i] += 1
    if place == "in place":
        h2, ring2, pos2 = s.h, ring, pos
    else:
        h2, ring2, pos2 = torch.full_like(s.h, 7.0), torch.full_like(ring, 7.0), torch.full_like(pos, 7)
    abi.mamba2_tree_commit(s.h, ring, pos, h2, ring2, pos2, xbc, xbc.stride(0), s.u, s.u.stride(0), s.dt, s.dt.stride(0),
                           s.A_log, s.dt_bias, cu, ints(flat), count, H, P, N, G, K)
    assert torch.equal(h2, h1) and torch.equal(ring2, ring1) and torch.equal(pos2, pos1)


def test_commit_follows_the_formula():
    H, P, N, G = 8, 64, 128, 2
    parents = [list(range(-1, 63))]
    s = Ssm(1, 64, H, P, N, G, 5)
    x, B, _ = s.parts()
    dt, dA = ref.steps(s.dt, s.dt_bias, s.A_log)
    path = list(range(64))
    want, size = s.h[0].to(ref.F), s.h[0].to(ref.F).abs()
    for r in path:
        want, size = ref.ssm_step(want, x[r], B[r], dt[r], dA[r]), ref.ssm_step(size, x[r].abs(), B[r].abs(), dt[r], dA[r])
    ring, pos = rows(3, s.W, gen(1)).view(1, 3, s.W), ints([0])
    out = torch.empty_like(s.h)
    abi.mamba2_tree_commit(s.h, ring, pos, out, ring, pos, s.u, s.u.stride(0), s.u, s.u.stride(0), s.dt, s.dt.stride(0),
                           s.A_log, s.dt_bias, [0, 64], ints(path), ints([64]), H, P, N, G, 4)
    # 64 steps of two roundings, and the factors' own
    close(out[0], want, 2.0 ** -15 * size)
    assert parents


def test_commit_reports_what_names_no_node():
    s = Ssm(2, 6, 2, 8, 16, 1, 6)
    ring, pos = rows(6, s.W, gen(1)).view(2, 3, s.W), ints([4, 4])
    h0, ring0 = s.h.clone(), ring.clone()

    def commit(path, count):
        out = s.h.clone(), ring.clone(), pos.clone()
        abi.mamba2_tree_commit(s.h, ring, pos, *out, s.u, s.u.stride(0), s.u, s.u.stride(0), s.dt, s.dt.stride(0), s.A_log,
                               s.dt_bias, [0, 3, 6], ints(path), ints(count), 2, 8, 16, 1, 4)
        return out
    good = commit([0, 1, -1, 0, 2, -1], [2, 2])
    assert abi.m2_device_status() == abi.M2_OK
    for path, count in (([0, 1, -1, 0, 3, -1], [2, 2]), ([0, 1, -1, 0, -5, -1], [2, 2]), ([0, 1, -1, -1, -1, -1], [2, -1]),
                        ([0, 1, -1, 0, 1, 2], [2, 4])):
        out = commit(path, count)
        assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
        assert all(torch.equal(a[0], b[0]) for a, b in zip(out, good))  # the other sequence
    assert torch.equal(s.h, h0) and torch.equal(ring, ring0)


# ------------------------------------------------------------------ verification

def verify(p, q, cu, parents, token, u, u_next, ld=None, stream=None):
    n, T, V = len(cu) - 1, cu[-1], p.shape[1]
    path, count, last = (_empty((k,), torch.int32, "cuda") for k in (max(T, 1), n, n))
    for t in (path, count, last):
        t.fill_(77)
    fmt = abi.M2_PROB_BF16 if p.dtype == bf else abi.M2_PROB_F32
    abi.m2_verify_tree(p, p.stride(0), q, 0 if q is None else q.stride(0), fmt, V, cu, ints([x for t in parents for x in t]),
                       ints(token), u, u_next, path, count, last, stream)
    return path[:T].tolist(), count.tolist(), last.tolist()


def same_as_reference(p, q, cu, parents, token, u, u_next):
    got = verify(p, q, cu, parents, token, u, u_next)
    ul, un = u.tolist(), u_next.tolist()
    path, count, last = [], [], []
    for i, t in enumerate(parents):
        a, b = cu[i], cu[i + 1]
        w, x = ref.verify(p[a:b], None if q is None else q[a:b], t, token[a:b], ul[a:b], un[i])
        path += w + [-1] * (b - a - len(w))
        count.append(len(w))
        last.append(x)
    assert got == (path, count, last)
    return got


def random_case(lens, V, kind, draft, seed, dtype=torch.float32, extra=0, close_to=0.5):
    g, T = gen(seed), sum(lens)
    parents, cu = trees(lens, kind, seed), offsets(lens)
    logits = 2.0 * torch.randn(max(T, 1), V, device="cuda", generator=g)
    q = torch.softmax(logits + close_to * torch.randn(max(T, 1), V, device="cuda", generator=g), -1)
    p = torch.softmax(logits, -1)
    above = [cu[i] + max(x, 0) for i, t in enumerate(parents) for x in t]
    token = torch.multinomial(q[above], 1, generator=g)[:, 0].tolist() if T else []
    if draft is None:  # children that differ: the most likely ones of the draft, in order
        rank = {}
        for i, t in enumerate(parents):
            for r, x in enumerate(t):
                k = rank[i, x] = rank.get((i, x), -1) + 1
                token[cu[i] + r] = int(q[cu[i] + max(x, 0)].topk(min(V, k + 1)).indices[-1])

    def wide(t):
        buf = _empty((len(t), V + extra), dtype, "cuda")
        buf.fill_(3.0)
        buf[:, extra:].copy_(t)
        return buf[:, extra:]
    return (wide(p), None if draft is None else wide(q), cu, parents, token, torch.rand(max(T, 1), device="cuda", generator=g),
            torch.rand(len(lens), device="cuda", generator=g))


@pytest.mark.parametrize("V", [1, 2, 7, 100, 1000, 16384, 16385, 50257, 131072])
@pytest.mark.parametrize("lens,kind", [([1], "chain"), ([5, 0, 9], "tree"), ([64, 2], "tree"), ([8, 8, 8], "star"),
                                       ([12], "chain")])
@pytest.mark.parametrize("draft", ["rows", None])
def test_verify(V, lens, kind, draft):
    for seed in range(3):
        same_as_reference(*random_case(lens, V, kind, draft, seed + V, extra=seed))


@pytest.mark.parametrize("extra", [0, 1, 4])
@pytest.mark.parametrize("draft", ["rows", None])
def test_verify_bf16_rows(extra, draft):
    for seed in range(4):
        same_as_reference(*random_case([7, 30], 4001, "star", draft, seed, dtype=bf, extra=extra, close_to=2.0))


def test_verify_many_sequences():
    same_as_reference(*random_case([1, 4, 0, 7] * 50, 300, "tree", "rows", 5))  # more than one launch takes


def test_verify_every_outcome():
    """Random numbers that force each branch: all accepted, all refused, the last token, the first."""
    p, q, cu, parents, token, u, u_next = random_case([20, 20], 5000, "star", "rows", 3, close_to=3.0)
    for uv in (0.0, 1.0 - 2.0 ** -24):
        for nv in (0.0, 0.5, 1.0 - 2.0 ** -24):
            u.fill_(uv)
            u_next.fill_(nv)
            path, count, _ = same_as_reference(p, q, cu, parents, token, u, u_next)
            if uv == 0.0:
                assert count == [2, 2] and path[:2] == [0, 1]


def test_verify_rows_that_leave_nothing():
    V = 600
    p = torch.zeros(4, V, device="cuda")
    p[0, 5], p[0, 9], p[1, 7] = 0.5, 0.5, 1.0
    q = p.clone()
    u = torch.full((4,), 1.0 - 2.0 ** -24, device="cuda")
    un = torch.tensor([0.75], device="cuda")
    # the draft is the target: accepted; a token without probability: refused, then nothing is left and the target serves
    assert verify(p, q, [0, 4], [[-1, 0, 1, 2]], [0, 5, 7, 3], u, un) == ([0, 1, 2, -1], [3], [-1])  # an empty row
    assert verify(p, q, [0, 2], [[-1, 0]], [0, 6], u[:2], un) == ([0, -1], [1], [9])
    # refused until one token is left, then that is refused too
    assert verify(p, None, [0, 3], [[-1, 0, 0]], [0, 5, 9], u[:3], un) == ([0, 2, -1], [2], [-1])
    u[2] = 2.0  # not a number in [0, 1): refused
    assert verify(p, None, [0, 3], [[-1, 0, 0]], [0, 5, 9], u[:3], un) == ([0, -1, -1], [1], [9])


def test_verify_odd_inputs():
    V = 1000
    p, q, cu, parents, token, u, u_next = random_case([9, 3, 1], V, "star", "rows", 8, close_to=2.0)
    for x in (float("nan"), float("inf"), -1.0, float("-inf")):
        p[0, 17], q[0, 18], p[3, V - 1], q[9, 0] = x, x, x, x
        token[2], token[3], token[4] = 17, 18, -1
        token[5] = V
        same_as_reference(p, q, cu, parents, token, u, u_next)
    parents[0][0], parents[1] = 0, [-1, -2, 5]  # no root; places without a node
    got = same_as_reference(p, q, cu, parents, token, u, u_next)
    assert got[1][0] == 0 and got[2][0] == -1 and got[0][:9] == [-1] * 9
    for t in (u, u_next):
        t.fill_(float("nan"))
    assert verify(p, q, cu, parents, token, u, u_next)[1] == [0, 1, 1]


def test_verify_far_rows():
    """Row offsets past 2^32 bytes."""
    V, T = 70000, 17
    ld = (5 << 30) // (4 * 16)  # row 16 begins at 5 GB
    buf = torch.empty(16 * ld + V, device="cuda")
    p = buf.as_strided((T, V), (ld, 1))
    small = torch.softmax(torch.randn(T, V, device="cuda", generator=gen(2)), -1)
    p.copy_(small)
    parents, u = [list(range(-1, T - 1))], torch.zeros(T, device="cuda")
    token = [0] * T
    got = verify(p, None, [0, T], parents, token, u, torch.tensor([0.3], device="cuda"))
    assert got == verify(small, None, [0, T], parents, token, u, torch.tensor([0.3], device="cuda"))
    assert got[1] == [T]


# ------------------------------------------------------------------ kept cache rows

@pytest.mark.parametrize("D,Hkv", [(128, 3), (64, 2)])
@pytest.mark.parametrize("past", [0, 1, 50, 61, 64, 127])
def test_keep(D, Hkv, past):
    lens = [64, 1, 0, 9, 40]
    parents, cu = trees(lens, "tree", past), offsets(lens)
    pasts = [past, 5, 70, past + 1, past + 30]
    c = Cache([a + b for a, b in zip(lens, pasts)], Hkv, D, past)
    picked, flat = paths_of(parents, random.Random(past))
    before = c.pages.clone()
    abi.m2_kv4_keep(c.struct, cu, ints(flat), ints([len(p) for p in picked]), ints(pasts))

    def bytes_of(pages, i, t):
        """Codes (a byte each) and scale bytes of a token, by the layout's formulas: [Hkv][...]."""
        pg, t = pages[int(c.table[i, t // 64])], t % 64
        v = pg[:, 32 * D + t // 8 * 4 * D:][:, :4 * D].reshape(Hkv, 8, 4, D // 8)[:, :, t % 8 // 2]
        vs = pg[:, 68 * D + t // 2 * (D // 8):][:, :D // 8].reshape(Hkv, D // 32, 2, 2)[:, :, t % 2]
        return (pg[:, t * (D // 2):(t + 1) * (D // 2)], (v >> (4 * (t % 2))) & 15,
                pg[:, 64 * D + t * (D // 16):][:, :D // 16], vs)
    for i, path in enumerate(picked):
        source = list(range(pasts[i] + lens[i]))
        for j, r in enumerate(path):
            source[pasts[i] + j] = pasts[i] + r
        for t, s in enumerate(source):
            for a, b in zip(bytes_of(c.pages, i, t), bytes_of(before, i, s)):
                assert torch.equal(a, b), (i, t, s)
    used = torch.zeros(c.n_pages, dtype=torch.bool, device="cuda")
    used[c.table[c.table >= 0].long()] = True
    assert torch.equal(c.pages[~used], before[~used])


def test_keep_leaves_out_and_reports():
    c = Cache([70, 70], 2, 64, 1)
    before = c.pages.clone()
    idle = abi.M2_KV4_IDLE
    path = ints([0, 3, 5, 7, -1, -1, -1, -1] * 2)

    def keep(counts, pos, path=path):
        c.pages.copy_(before)
        abi.m2_kv4_keep(c.struct, [0, 8, 16], path, ints(counts), ints(pos))
        return abi.m2_device_status(clear=True)
    assert keep([4, 4], [idle, idle]) == abi.M2_OK and torch.equal(c.pages, before)
    assert keep([0, 1], [60, 60]) == abi.M2_OK and torch.equal(c.pages, before)
    assert keep([4, 0], [-5, 60]) == abi.M2_ERR_ARG and torch.equal(c.pages, before)
    assert keep([4, 0], [128, 60]) == abi.M2_ERR_ARG and torch.equal(c.pages, before)
    assert keep([4, -3], [60, 60]) == abi.M2_ERR_ARG
    one = c.pages.clone()
    assert keep([4, 0], [60, 60]) == abi.M2_OK and torch.equal(c.pages, one) and not torch.equal(one, before)
    assert keep([4, 0], [60, 60], ints([0, 3, 99, 7, -1, -1, -1, -1] * 2)) == abi.M2_ERR_ARG
    c.table[0, 1] = c.n_pages  # the page of tokens 64 .. : source of 65 (60 + 5) and 67
    assert keep([4, 0], [60, 60]) == abi.M2_ERR_ARG
    c.table[0, 1] = -1
    assert keep([2, 0], [60, 60]) == abi.M2_OK  # 63 -> 61 needs the first page only


# ------------------------------------------------------------------ attention

def run_tree(lens, pasts, H, Hkv, D, kind="tree", seed=0, spread=1.0, vspread=1.0, scale=None, fix=None, width=None,
             extra=0, parents=None, q_fix=None):
    g = gen(seed + H + D)
    parents = parents or trees(lens, kind, seed)
    cu, T, ends = offsets(lens), sum(lens), [a + b for a, b in zip(lens, pasts)]
    c = Cache(ends, Hkv, D, seed, width=width)
    ce = offsets(ends)
    k, v = rows(ce[-1], Hkv * D, g), rows(ce[-1], Hkv * D, g, spread=vspread)
    if fix:
        fix(k.view(-1, Hkv, D), v.view(-1, Hkv, D), ce)
    c.append(k, v, ce, [0] * len(lens))
    q = rows(T, H * D, g, extra, spread)
    if q_fix:
        q_fix(q)
    buf, out = out_rows(T, H * D, extra)
    scale = D ** -0.5 if scale is None else scale
    ws = _empty((abi.m2_attn_tree_kv4_workspace_bytes(H, Hkv, D),), torch.uint8, "cuda")
    ws.fill_(0xFF)  # (NaN wherever it is read unwritten)
    abi.m2_attn_tree_kv4(c.struct, q, q.stride(0), out, out.stride(0), H, cu, ints([p for t in parents for p in t]),
                         ints(pasts), scale, ws, ws.numel())
    assert bool((buf[:, :extra] == 7).all())
    kk, vv = (attention_ref.rounded_rows(t.reshape(-1, Hkv, D)) for t in (k, v))
    for i, t in enumerate(parents):
        r, e = slice(cu[i], cu[i + 1]), slice(ce[i], ce[i + 1])
        want, size, total, score = ref.attend(q[r].reshape(-1, H, D), kk[e], vv[e], scale, pasts[i], t)
        close(out[r].reshape(-1, H, D), want,
              BF16 * want.abs() + (F16 + EVAL + 2.0 ** -19 * score) * size + 2.0 ** -32 * total + 1e-30)
    return c, q, out, (cu, parents, pasts, ws, scale)


HEADS = [(32, 8, 128), (4, 4, 128), (7, 1, 128), (8, 2, 64), (3, 3, 64), (20, 1, 64), (24, 2, 128)]


@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("kind", ["chain", "tree", "star", "forest"])
def test_attention_lengths_and_heads(H, Hkv, D, kind):
    run_tree([1, 0, 5, 16], [0, 9, 64, 200], H, Hkv, D, kind, extra=8)
    run_tree([64, 3], [61, 700], H, Hkv, D, kind, seed=1)


@pytest.mark.parametrize("lens,pasts,H,Hkv,D", [
    ([4], [131], 32, 8, 128), ([8], [5000], 32, 8, 128), ([16], [20000], 4, 1, 128), ([3] * 40, [70 * i for i in range(40)], 8, 2, 64),
    ([64, 64], [3000, 64], 32, 8, 128), ([1] * 130, [i for i in range(130)], 4, 2, 128), ([33, 1, 64, 0, 2], [0, 0, 1, 5, 8000], 16, 2, 64),
    ([7], [30000], 64, 1, 64)])
@pytest.mark.parametrize("width", [None, 600])
def test_attention_splits(lens, pasts, H, Hkv, D, width):
    run_tree(lens, pasts, H, Hkv, D, seed=2, width=width)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("past", list(range(0, 130, 13)) + [63, 64, 127, 128])
def test_attention_trees_at_page_borders(D, past):
    run_tree([64, 17, 2], [past, past, past], 4, 2, D, "forest", seed=past)


def test_attention_padded_places():
    parents = [[-1, 0, -2, 2, 1, 4, 9, -1], [-1] + [-2] * 30, [-2, 0, 1], [-3]]
    _, _, out, _ = run_tree([8, 31, 3, 1], [70, 10, 0, 64], 8, 2, 128, parents=parents)
    for r in (2, 3, 6, *range(9, 39), 39, 40, 41, 42):
        assert bool((out[r] == 0).all())


@pytest.mark.parametrize("spread,vspread", [(30.0, 1.0), (1e4, 300.0), (1e-6, 1e-3)])
def test_attention_ranges(spread, vspread):
    run_tree([9, 30], [100, 300], 8, 2, 128, spread=spread if spread > 1 else 1.0, vspread=vspread,
             scale=1e-4 if spread > 100 else None)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_attention_scales(scale):
    run_tree([9, 30], [100, 3], 8, 2, 64, scale=scale)


def test_attention_scores_that_grow():
    def fix(k, v, ce):
        k.mul_(torch.linspace(0.0, 4.0, k.shape[0], device="cuda").view(-1, 1, 1).to(bf))
    run_tree([20], [1500], 8, 2, 128, fix=fix, spread=3.0)


@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (32, 2, 64), (2, 2, 64)])
@pytest.mark.parametrize("past", [0, 60, 64, 130])
@pytest.mark.parametrize("what", ["k", "v"])
def test_attention_bad_values_reach_only_the_nodes_below(H, Hkv, D, past, what):
    """A node's NaN key or value, and what lies behind the last node."""
    parents, at = [[-1, 0, 0, 1, 2, 3, 1, 6, 4, 4]], 6
    n = len(parents[0])
    good = run_tree([n], [past], H, Hkv, D, parents=parents)

    def fix(k, v, ce):
        (k if what == "k" else v)[past + at, 0, 5] = float("nan")
    g = gen(H + D)
    c = Cache([past + n], Hkv, D, 0)
    k, v = rows(past + n, Hkv * D, g), rows(past + n, Hkv * D, g)
    fix(k.view(-1, Hkv, D), v.view(-1, Hkv, D), None)
    c.append(k, v, [0, past + n], [0])
    q = rows(n, H * D, g)
    out = torch.empty_like(q)
    cu, parents, pasts, ws, scale = good[3]
    abi.m2_attn_tree_kv4(c.struct, q, H * D, out, H * D, H, cu, ints(parents[0]), ints(pasts), scale, ws, ws.numel())
    o, w = out.view(n, H, D), good[2].reshape(n, H, D)
    hit = [r for r, p in enumerate(ref.paths(parents[0])) if at in p]
    other = [r for r in range(n) if r not in hit]
    assert torch.equal(o[other], w[other])
    G = H // Hkv
    assert torch.equal(o[:, G:], w[:, G:])  # the other kv heads
    assert bool(o[hit][:, :G, :16].isnan().all())
    if what == "v":  # a group of 16 channels is NaN, as the cache holds it
        off = (o[hit][:, :G, 16:].float() - w[hit][:, :G, 16:].float()).abs()
        assert bool((off <= 0.05 * w.float().abs().max()).all())
    else:
        assert bool(o[hit][:, :G].isnan().all())


def test_attention_left_out_and_reported():
    H, Hkv, D = 8, 2, 128
    c, q, out, (cu, parents, pasts, ws, scale) = run_tree([4, 4, 4], [124, 60, 10], H, Hkv, D, "chain", width=2)  # the first fills its table
    flat = ints([p for t in parents for p in t])

    def run(pos):
        o = torch.full_like(out, 7.0)
        abi.m2_attn_tree_kv4(c.struct, q, q.stride(0), o, o.stride(0), H, cu, flat, ints(pos), scale, ws, ws.numel())
        return o, abi.m2_device_status(clear=True)
    o, st = run([abi.M2_KV4_IDLE, 60, abi.M2_KV4_IDLE])
    assert st == abi.M2_OK and bool((o[:4] == 0).all()) and bool((o[8:] == 0).all()) and torch.equal(o[4:8], out[4:8])
    o, st = run([124, 60, -1])
    assert st == abi.M2_ERR_ARG and bool((o[8:] == 0).all()) and torch.equal(o[:8], out[:8])
    o, st = run([126, 60, 10])  # the last two nodes lie past the table's 128 tokens
    assert st == abi.M2_ERR_ARG and torch.equal(o[4:], out[4:]) and bool(o[:4].isfinite().all())
    o, st = run([2 ** 31 - 1, 60, 10])
    assert st == abi.M2_ERR_ARG and torch.equal(o[4:], out[4:])
    saved = int(c.table[1, 0])
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        c.table[1, 0] = bad  # all of the sequence's context: what is left are its nodes
        o, st = run([124, 64, 10])
        assert st == abi.M2_ERR_ARG and torch.equal(o[:4], out[:4]) and torch.equal(o[8:], out[8:])
    c.table[1, 0] = saved
    assert torch.equal(run([124, 60, 10])[0], out)


def test_attention_infinite_queries_give_zeros_or_nan_as_single_tokens_do():
    def q_fix(q):
        q[2, 3] = float("inf")
    H, Hkv, D = 4, 2, 64
    c, q, _, (cu, parents, pasts, ws, scale) = run_tree([5], [70], H, Hkv, D, "chain")
    base = torch.empty_like(q)
    q_fix(q)
    abi.m2_attn_tree_kv4(c.struct, q, H * D, base, H * D, H, cu, ints(parents[0]), ints(pasts), scale, ws, ws.numel())
    one = torch.empty(1, H * D, dtype=bf, device="cuda")
    w2 = torch.empty(abi.m2_attn_decode_kv4_workspace_bytes(1, H, Hkv, D), dtype=torch.uint8, device="cuda")
    abi.m2_attn_decode_kv4(c.struct, q[2:3], H * D, one, H * D, H, ints([73]), scale, w2, w2.numel())
    assert torch.equal(one[0].isnan(), base[2].isnan())
    assert bool(base[[0, 1, 3, 4]].isfinite().all())


def test_attention_is_deterministic_and_repeats():
    c, q, out, (cu, parents, pasts, ws, scale) = run_tree([30, 64, 9], [4000, 100, 2000], 32, 8, 128, width=100)
    for _ in range(5):
        o = torch.empty_like(out)
        abi.m2_attn_tree_kv4(c.struct, q, q.stride(0), o, o.stride(0), 32, cu, ints([p for t in parents for p in t]),
                             ints(pasts), scale, ws, ws.numel())
        assert torch.equal(o, out)
