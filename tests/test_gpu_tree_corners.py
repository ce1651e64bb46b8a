"""Faults that were found in the operators for trees of drafted tokens, each held by what it
answered wrongly.  Plain forms in tree_ref.py."""
import random

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from tests import tree_ref as ref
from tests.test_gpu_attention import gen, rows
from tests.test_gpu_tree import Ssm, ints, same_as_reference, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


# ------------------------------------------------------------------ verification: what refused tokens leave

def row(V, values):
    p = torch.zeros(1, V, device="cuda")
    for x, v in values.items():
        p[0, x] = v
    return p


def floats(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


BELOW_ONE = 1.0 - 2.0 ** -24


def test_verify_draws_the_little_that_refused_tokens_leave():
    """Two tokens hold all but 5e-8 of the row: they are refused, and the third is drawn."""
    for at in ([0, 1, 2], [0, 1, 999], [999, 0, 1], [5, 400, 700]):
        p = row(1000, dict(zip(at, (0.4566476, 0.54335237, 4.7786124e-8))))
        p = p.expand(3, -1).contiguous()
        got = verify(p, None, [0, 3], [[-1, 0, 0]], [0, at[0], at[1]], floats(0.0, 0.9, BELOW_ONE), floats(0.5))
        assert got == ([0, -1, -1], [1], [at[2]])


@pytest.mark.parametrize("V", [3, 40, 1000, 70000])
@pytest.mark.parametrize("u_next", [0.0, 0.5, BELOW_ONE, 1.0])
def test_verify_never_draws_a_refused_token(V, u_next):
    """Runs that hold refused tokens alone, beside one with a token that is left; a random number of 1 takes the last."""
    rng = random.Random(V)
    for n in (2, 5, 40):
        n = min(n, V - 1)
        far = sorted(rng.sample(range(V), n + 1))
        left = far.pop(rng.randrange(n + 1))
        weight = (torch.rand(n, generator=torch.Generator().manual_seed(n)) + 0.1).tolist()
        p = row(V, {x: w / sum(weight) for x, w in zip(far, weight)})
        p[0, left] = 2.0 ** -40
        p = p.expand(n + 1, -1).contiguous()
        u = torch.full((n + 1,), 2.0, device="cuda")  # (refused whatever is left)
        got = verify(p, None, [0, n + 1], [[-1] + [0] * n], [0] + far, u, floats(u_next))
        assert got == ([0] + [-1] * n, [1], [left]), n


@pytest.mark.parametrize("V", [64, 5000])
def test_verify_refused_tokens_beside_values_that_are_none(V):
    """Infinities and NaN in the same run as refused tokens."""
    p = row(V, {3: 0.25, 9: 0.25, 11: 0.5, 20: float("inf"), 21: float("nan"), 22: -1.0}).expand(4, -1).contiguous()
    for un in (0.0, 0.4, BELOW_ONE):
        same_as_reference(p, None, [0, 4], [[-1, 0, 0, 0]], [0, 11, 3, 20], floats(0.0, 0.9, BELOW_ONE, 0.0), floats(un))


# ------------------------------------------------------------------ SSM outputs: rows far apart

def test_ssm_rows_of_many_channels():
    """56 rows of H * P outputs pass 2^31 elements: what the first, middle and last heads give alone."""
    H, P, N, G, n = 150016, 256, 16, 1, 64
    assert 56 * H * P > 2 ** 31
    g = gen(1)
    h = torch.empty(1, H, P, N, device="cuda").normal_(generator=g)
    x = torch.empty(n, H * P, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    bc, dt = rows(n, 2 * N, g), rows(n, H, g)
    A_log, D, bias = (torch.rand(H, device="cuda", generator=g) for _ in range(3))
    parent = ints(ref.random_parents(n, random.Random(1)))
    wide = torch.empty(n, 2, H * P, dtype=torch.bfloat16, device="cuda")  # B and C at x's stride
    wide[:, 0, :2 * N].copy_(bc)
    B, C, ld = wide[:, 0], wide[:, 0, N:], 2 * H * P
    wide[:, 1].copy_(x)
    del x
    x, y = wide[:, 1], torch.full((n, H * P), 7.0, device="cuda")
    abi.mamba2_tree_ssm(h, x, B, C, ld, dt, H, A_log, D, bias, y, [0, n], parent, H, P, N, G)
    for h0 in (0, H // 2, H - 8):
        one, to = torch.empty(n, 8 * P, device="cuda"), slice(h0, h0 + 8)
        abi.mamba2_tree_ssm(h[0, to], x[:, h0 * P:], B, C, ld, dt[:, h0:], H, A_log[to].clone(), D[to].clone(), bias[to].clone(),
                            one, [0, n], parent, 8, P, N, G)
        assert torch.equal(y[:, h0 * P:(h0 + 8) * P], one)


# ------------------------------------------------------------------ commit: shared memory next to what needs no asking

@pytest.mark.parametrize("N,n", [(16, 46), (16, 45), (16, 47), (32, 45), (32, 44), (32, 46)])
@pytest.mark.parametrize("G", [1, 2])
def test_commit_of_wide_heads(N, n, G):
    """Heads of 256 channels, enough of them for the longest blocks, and paths whose inputs just fill the shared memory
    that a kernel has without asking for more (of which a block's own arrays take 768 bytes)."""
    H, P, K, B = 40, 256, 4, 8
    s = Ssm(B, B * n, H, P, N, G, n, extra=4)
    W, xbc = s.W, s.u.contiguous() if G == 1 else s.u  # (in one launch; with the ring in a launch of its own)
    ring, pos = rows(B * (K - 1), W, gen(2)).view(B, K - 1, W), ints([7 * i for i in range(B)])
    h1, ring1, pos1 = s.h.clone(), ring.clone(), pos.clone()
    for j in range(n):
        u, dt = s.u[j::n].contiguous(), s.dt[j::n].contiguous()
        dt = torch.cat([dt, dt.new_zeros(B, W - H)], 1)
        y = torch.empty(B, H * P, device="cuda")
        abi.mamba2_ssm_step(h1, u, u[:, H * P:], u[:, H * P + G * N:], dt, W, s.A_log, s.D, s.dt_bias, y, B, H, P, N, G)
        ring1[torch.arange(B, device="cuda"), (pos1 % (K - 1)).long()] = s.u[j::n]
        pos1 += 1
    abi.mamba2_tree_commit(s.h, ring, pos, s.h, ring, pos, xbc, xbc.stride(0), s.u, s.u.stride(0), s.dt, s.dt.stride(0),
                           s.A_log, s.dt_bias, [n * i for i in range(B + 1)], ints(list(range(n)) * B), ints([n] * B), H, P,
                           N, G, K)
    assert torch.equal(s.h, h1) and torch.equal(ring, ring1) and torch.equal(pos, pos1)


# ------------------------------------------------------------------ verification: tokens whose remainder is next to 0

def bits(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda").view(torch.float32)


def test_verify_remainders_next_to_zero():
    """After two refusals c q of token 0 is its p but for half a rounding, which is 2^-16 of what all leave together and
    moves the third child's comparison."""
    q = bits(0x3f000000, 0x3e999998, 0x3d4ccccd, 0x3e19999a)
    p = bits(0x3f066668, 0x3ea18937, 0, 0x3e2353f8)
    P, Q = p.to(ref.F), q.to(ref.F)
    c = 1 + (P - Q).clamp(min=0).sum()
    left = (P - c * Q).clamp(min=0)
    border = float(left[1] / (Q[1] * left.sum()))
    assert 0 < float(left[0]) < 2.0 ** -24 * float(P[0]) and 0 < border < 1
    for V in (4, 3000):
        pr, qr = torch.zeros(4, V, device="cuda"), torch.zeros(4, V, device="cuda")
        pr[:, :4], qr[:, :4] = p, q
        for off in (-4e-6, -1e-6, -2e-7, 2e-7, 1e-6, 4e-6):
            u = floats(0.0, 0.9, 0.9, border + off)
            for un in (0.0, 0.1, 0.25, 0.9):
                got = same_as_reference(pr, qr, [0, 4], [[-1, 0, 0, 0]], [0, 2, 2, 1], u, floats(un))
                assert (got[1] == [2]) == (off < 0)


# ------------------------------------------------------------------ calls without nodes

@pytest.mark.parametrize("P", [64, 3])
def test_commit_without_nodes(P):
    """No array by node: outputs apart are written whole, what is in place stays."""
    H, N, G, K, B = 1, 16, 1, 4, 3
    s = Ssm(B, 1, H, P, N, G, 1)
    ring, pos = rows(B * (K - 1), s.W, gen(2)).view(B, K - 1, s.W), ints([5, 6, 7])
    count = ints([0] * B)
    before = s.h.clone(), ring.clone(), pos.clone()
    out = torch.full_like(s.h, 7.0), torch.full_like(ring, 7.0), torch.full_like(pos, 7)
    for o in (out, (s.h, ring, pos)):
        launches = abi.m2_launch_count()
        abi.mamba2_tree_commit(s.h, ring, pos, *o, None, 0, None, 0, None, 0, s.A_log, s.dt_bias, [0] * (B + 1), None, count,
                               H, P, N, G, K)
        assert all(torch.equal(a, b) for a, b in zip(o, before))
        assert (abi.m2_launch_count() == launches) == (o[0] is s.h)


def test_verify_without_nodes():
    count, last = ints([7] * 3), ints([7] * 3)
    abi.m2_verify_tree(None, 0, None, 0, abi.M2_PROB_F32, 100, [0] * 4, None, None, None, floats(0.1, 0.2, 0.3), None, count, last)
    assert count.tolist() == [0] * 3 and last.tolist() == [-1] * 3


# ------------------------------------------------------------------ conv: outputs beside its inputs

def test_conv_into_other_columns_of_its_rows():
    g, C, K, n = gen(4), 64, 4, 9
    ring, w, b = rows(3, C, g).view(1, 3, C), rows(C, K, g), rows(1, C, g)[0]
    parent = ints(ref.random_parents(n, random.Random(2)))
    for left in (True, False):
        both = rows(n, 2 * C, g)
        x, out = (both[:, :C], both[:, C:]) if left else (both[:, C:], both[:, :C])
        before = x.clone()
        apart = torch.empty(n, C, dtype=x.dtype, device="cuda")
        abi.mamba2_tree_conv(ring, ints([5]), x, 2 * C, w, b, apart, C, [0, n], parent, C, K)
        abi.mamba2_tree_conv(ring, ints([5]), x, 2 * C, w, b, out, 2 * C, [0, n], parent, C, K)
        assert torch.equal(out, apart) and torch.equal(x, before)


# ------------------------------------------------------------------ SSM outputs: decays without bound

@pytest.mark.parametrize("n", [5, 30, 64])
def test_ssm_decays_that_overflow(n):
    """dt A below fp32's range: a step keeps nothing of what was before it, and its own term whole."""
    parents = [ref.random_parents(n, random.Random(n), "forest")]
    s = Ssm(1, n, 6, 16, 32, 2, 4, extra=4)
    s.A_log[0], s.A_log[1], s.A_log[2], s.A_log[3] = 90.0, float("inf"), 75.0, -float("inf")
    s.dt[1::3, 2] = float("inf")  # a step of 1e9
    y = s.run([0, n], parents).view(n, 6, 16)
    x, B, C = s.parts()
    want, size = ref.ssm(s.h[0], x, B, C, s.dt, s.dt_bias, s.A_log, s.D, parents[0])
    assert bool(want.isfinite().all()) and bool(y.isfinite().all())
    decay = torch.log(ref.steps(s.dt, s.dt_bias, s.A_log)[1])  # of the paths, as far as any of it is left
    path = ref.ancestors_sum(parents[0], decay).abs().clamp(max=200.0)[..., None]
    assert bool(((y - want).abs() <= (2.0 ** -17 + path * 2.0 ** -21) * size + 1e-30).all())
    s.A_log[4] = float("nan")
    assert bool(s.run([0, n], parents).view(n, 6, 16)[:, 4].isnan().all())
