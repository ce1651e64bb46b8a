"""The attention operators against their 64-bit plain forms.

Tolerances count roundings.  A value rounded to bf16 is off by at most 2^-8 of
itself (half a step), to f16 by 2^-11.  fp32 evaluation adds EVAL of the sum of
magnitudes: products and sums over at most 128 channels with scores of a few
units put an error of about 2^-24 * 128 on a score, and the exponentials about
2^-22, together below 2^-15 relative on a probability.  Attention: the
probabilities' rounding (PREC) and EVAL scale with sum p |v|, the output's
rounding with the output."""
import math

import pytest
import torch

from mamba_ssm_layer_gb300 import abi
from mamba_ssm_layer_gb300.layer import _empty
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = 2.0 ** -8, 2.0 ** -11
EVAL = 2.0 ** -15
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(T, width, g, extra=0, spread=1.0):
    """[T][width] bf16 rows, `extra` elements between them (a column range of wider rows when extra > 0)."""
    buf = _empty((max(T, 1), width + extra), bf, "cuda")
    buf.copy_(torch.randn(max(T, 1), width + extra, device="cuda", generator=g) * spread)
    return buf[:T, extra:]


def out_rows(T, width, extra=0):
    buf = _empty((max(T, 1), width + extra), bf, "cuda")
    buf.fill_(7.0)
    return buf, buf[:T, extra:]


def close(got, want, tol):
    got = got.to(ref.F)
    same_nan = torch.equal(got.isnan(), want.isnan())
    assert same_nan, "NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    fine = want.isfinite()
    off = (got - want).abs()[fine]
    lim = tol[fine]
    bad = off > lim
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / lim).max()):.3g} of the tolerance"


# ------------------------------------------------------------------ head norm and rotation

@pytest.mark.parametrize("T,H,Hkv,D,rot,inter,norm", [
    (1, 32, 8, 128, 128, False, True), (64, 32, 8, 128, 128, False, True), (700, 4, 1, 128, 128, True, True),
    (5, 7, 1, 64, 64, False, True), (33, 3, 3, 64, 32, True, True), (2, 2, 1, 128, 16, False, False),
    (9, 1, 1, 64, 0, False, True), (1300, 6, 2, 64, 48, False, False), (17, 5, 5, 128, 96, False, True),
    (3, 2, 2, 128, 0, False, False)])
@pytest.mark.parametrize("form", ["apart", "strided", "in place"])
def test_rope(T, H, Hkv, D, rot, inter, norm, form):
    g = gen(T + H + D)
    extra = 8 * 5 if form == "strided" else 0
    q, k = rows(T, H * D, g, extra), rows(T, Hkv * D, g, extra, 3.0)
    q0, k0 = q.clone(), k.clone()
    q_w, k_w = (rows(1, D, g).view(-1).abs() + 0.5 for _ in range(2)) if norm else (None, None)
    pos = torch.randint(-5, 2 ** 31 - 1, (T,), device="cuda", generator=g, dtype=torch.int32)
    pos[: T // 2] = torch.arange(T // 2, device="cuda")
    theta = 500000.0 if rot == 96 else 10000.0
    steps = torch.tensor(abi.m2_rope_steps(theta, rot), dtype=torch.int64, device="cuda") if rot else None
    qo, ko = (q, k) if form == "in place" else (out_rows(T, H * D, extra)[1], out_rows(T, Hkv * D, extra)[1])
    abi.m2_qk_norm_rope(q, q.stride(0), k, k.stride(0), qo, qo.stride(0), ko, ko.stride(0), q_w, k_w,
                        pos if rot else None, steps, T, H, Hkv, D, rot, inter, 1e-5)
    for got, x, w, n in ((qo, q0, q_w, H), (ko, k0, k_w, Hkv)):
        # the far angle: a double's own product with the frequency is off by 2^-53 of up to 2^31 radians, and the
        # step's by as much
        y, size = ref.rope(x.view(T, n, D) if x.is_contiguous() else x.reshape(T, n, D), w, pos, theta, rot, inter, 1e-5)
        close(got.reshape(T, n, D), y, BF16 * y.abs() + (2.0 ** -20 + 2.0 ** -20) * size)


# ------------------------------------------------------------------ the 4-bit cache

class Cache:
    """A pool with random bytes in every slot, and pages of `lens` tokens a sequence in a random order."""

    def __init__(self, lens, Hkv, D, seed, spare=2, first_page=0, width=None):
        g = gen(seed)
        need = [-(-n // 64) for n in lens]
        total = sum(need) + spare
        self.Hkv, self.D, self.n_pages = Hkv, D, total + first_page
        self.pages = _empty((self.n_pages, Hkv, 72 * D), torch.uint8, "cuda")
        self.pages[first_page:].copy_(torch.randint(0, 256, (total, Hkv, 72 * D), device="cuda", generator=g,
                                                    dtype=torch.uint8))
        ids = (torch.randperm(total, device="cuda", generator=g) + first_page).tolist()
        width = width or max(1, max(need))
        table = [[-1] * width for _ in lens]
        for row, n in zip(table, need):
            for j in range(n):
                row[j] = ids.pop()
        self.table = _empty((len(lens), width), torch.int32, "cuda")
        self.table.copy_(torch.tensor(table, dtype=torch.int32))
        self.struct = abi.kv4_cache(self.pages, self.n_pages, Hkv, D, self.table, len(lens), width)

    def append(self, k, v, cu, past):
        p = torch.tensor(past, dtype=torch.int32, device="cuda")
        abi.m2_kv4_append(self.struct, k, k.stride(0), v, v.stride(0), cu, p)

    def gather(self, cu, extra=0):
        w = self.Hkv * self.D
        (kb, k), (vb, v) = out_rows(cu[-1], w, extra), out_rows(cu[-1], w, extra)
        abi.m2_kv4_gather(self.struct, k, k.stride(0) if len(k) else w + extra, v, v.stride(0) if len(v) else w + extra,
                          cu)
        if extra:
            assert bool((kb[:, :extra] == 7).all()) and bool((vb[:, :extra] == 7).all())
        return k, v


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("D,Hkv", [(128, 8), (128, 1), (64, 3), (64, 2)])
@pytest.mark.parametrize("calls", [
    [[1]], [[64, 0, 65]], [[3, 1, 0], [1, 0, 5], [1, 1, 1], [60, 64, 3], [1, 200, 129]],
    [[7] * 200, [1] * 200],  # more sequences than one launch takes
    [[1]] * 9])
def test_cache_append_and_gather(D, Hkv, calls):
    n = len(calls[0])
    ends = [sum(c[i] for c in calls) for i in range(n)]
    c = Cache(ends, Hkv, D, D + Hkv)
    g = gen(n)
    before = c.pages.clone()
    past, want_k, want_v = [0] * n, [[] for _ in range(n)], [[] for _ in range(n)]
    for lens in calls:
        cu = offsets(lens)
        k, v = rows(cu[-1], Hkv * D, g, 8), rows(cu[-1], Hkv * D, g, 16, 0.02)
        c.append(k, v, cu, past)
        rk, rv = ref.rounded_rows(k.reshape(-1, Hkv, D)), ref.rounded_rows(v.reshape(-1, Hkv, D))
        for i in range(n):
            want_k[i].append(rk[cu[i]:cu[i + 1]])
            want_v[i].append(rv[cu[i]:cu[i + 1]])
            past[i] += lens[i]
    cu = offsets(ends)
    k, v = c.gather(cu, extra=8)
    assert torch.equal(k.to(ref.F).reshape(-1, Hkv, D), torch.cat([torch.cat(x) for x in want_k]))
    assert torch.equal(v.to(ref.F).reshape(-1, Hkv, D), torch.cat([torch.cat(x) for x in want_v]))
    # pages that belong to nobody are as they were
    used = torch.zeros(c.n_pages, dtype=torch.bool, device="cuda")
    used[c.table[c.table >= 0].long()] = True
    assert torch.equal(c.pages[~used], before[~used])
    # a part of every sequence
    part = [m // 2 for m in ends]
    k2, _ = c.gather(offsets(part))
    for i in range(n):
        assert torch.equal(k2[offsets(part)[i]:offsets(part)[i + 1]], k[cu[i]:cu[i] + part[i]])


@pytest.mark.parametrize("D", [64, 128])
def test_cache_bytes(D):
    """The page's bytes are the documented ones, and slots past the last token keep theirs."""
    Hkv, n = 2, 41  # an odd end: the last pair's high nibbles
    c = Cache([n], Hkv, D, 5)
    page = int(c.table[0, 0])
    before = c.pages[page].clone().cpu()
    g = gen(1)
    k, v = rows(n, Hkv * D, g), rows(n, Hkv * D, g)
    c.append(k, v, [0, n], [0])
    got = c.pages[page].cpu()
    for h in range(Hkv):
        kc, kb = ref.quantize(k.view(n, Hkv, D)[:, h].cpu())
        vc, vb = ref.quantize(v.view(n, Hkv, D)[:, h].cpu())
        full = [torch.zeros(64, t.shape[1], dtype=torch.uint8) for t in (kc, kb, vc, vb)]
        mask = [torch.zeros(64, t.shape[1], dtype=torch.uint8) for t in (kc, kb, vc, vb)]
        for f, m, t in zip(full, mask, (kc, kb, vc, vb)):
            f[:n] = t
            m[:n] = 15 if f.shape[1] == D else 255
        # the sign of a zero code is not part of its value
        want, bits = ref.pack_block(*full), ref.pack_block(*mask)
        mine = got[h]
        zero = ~(((want & bits & 0x77) == (mine & bits & 0x77)) | (torch.arange(72 * D) >= 64 * D))
        assert not zero.any()
        code = torch.arange(72 * D) < 64 * D
        assert torch.equal(want[~code] & bits[~code], mine[~code] & bits[~code])
        untouched = bits == 0
        assert torch.equal(mine[untouched], before[h][untouched])


def test_cache_extreme_values():
    D, x = 128, torch.zeros(12, 128, device="cuda")
    x[0, :16] = torch.tensor([6.0, 0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, -5.0, 4.99, 5.01, 1e-3, -6.0, 0, 2])
    x[1, 3] = math.inf
    x[1, 20], x[1, 21] = -math.inf, 1.0
    x[2, 40] = math.nan
    x[2, 41] = 3.0
    x[3] = 1e30
    x[4] = -1e-30
    x[5] = torch.linspace(1e-6, 1e-4, 128)
    x[6] = torch.linspace(-61440, 70000, 128)
    x[7] = 2.0 ** -14 * 6
    x[8] = torch.arange(128) * 2.0 ** -17
    x[9] = 2.0 ** -133  # a bf16 subnormal
    g = gen(3)
    x[10:] = torch.exp2(torch.randint(-20, 16, (2, 128), device="cuda", generator=g).float()) * \
        torch.randn(2, 128, device="cuda", generator=g)
    x = x.to(bf)
    c = Cache([12], 1, D, 1)
    c.append(x, x, [0, 12], [0])
    k, v = c.gather([0, 12])
    want = ref.rounded_rows(x)
    assert bool(want[2, 32:48].isnan().all()) and not bool(want[2, :32].isnan().any())
    for got in (k, v):
        close(got, want, torch.zeros_like(want))


def test_cache_leaves_out_what_the_table_does_not_cover():
    Hkv, D = 2, 64
    c = Cache([200, 64, 10], Hkv, D, 2, width=4)
    good = c.table.clone()
    c.table[0, 1] = c.n_pages      # past the pool
    c.table[1, 0] = -7
    before = c.pages.clone()
    g = gen(4)
    lens = [200, 64, 10]
    k, v = rows(274, Hkv * D, g), rows(274, Hkv * D, g)
    abi.m2_device_status(clear=True)
    c.append(k, v, offsets(lens), [0, 0, 0])
    assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
    # the pages meant were not written, nor any page that is nobody's
    for page in (int(good[0, 1]), int(good[1, 0])):
        assert torch.equal(c.pages[page], before[page])
    kk, vv = c.gather(offsets(lens))
    assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
    want = ref.rounded_rows(k.view(-1, Hkv, D)).view(274, -1)
    keep = torch.ones(274, dtype=torch.bool, device="cuda")
    keep[64:128] = False
    keep[200:264] = False
    assert torch.equal(kk.to(ref.F)[keep], want[keep])
    assert bool((kk[~keep] == 7).all()) and bool((vv[~keep] == 7).all())
    # negative positions and positions past the table
    before = c.pages.clone()
    c.append(k[:20], v[:20], [0, 10, 10, 20], [250, 0, -20])
    assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
    changed = (c.pages != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(good[0, 3])]  # tokens 250 .. 255
    c.append(k[:1], v[:1], [0, 1, 1, 1], [0, 0, 0])
    assert abi.m2_device_status(clear=True) == abi.M2_OK


# ------------------------------------------------------------------ prompts

def run_prefill(lens_q, lens_k, H, Hkv, D, seed=0, extra=0, fix=None, scale=None, spread=1.0):
    g = gen(seed + sum(lens_q))
    cu_q, cu_k = offsets(lens_q), offsets(lens_k)
    q = rows(cu_q[-1], H * D, g, extra, spread)
    k, v = rows(cu_k[-1], Hkv * D, g, extra), rows(cu_k[-1], Hkv * D, g, extra)
    if fix:
        fix(q, k, v, cu_q, cu_k)
    scale = D ** -0.5 if scale is None else scale
    buf, out = out_rows(cu_q[-1], H * D, extra)
    abi.m2_attn_prefill_varlen(q, H * D + extra, k, Hkv * D + extra, v, Hkv * D + extra, out, H * D + extra, H, Hkv, D,
                               cu_q, cu_k, scale, torch.cuda.current_stream())
    if extra:
        assert bool((buf[:, :extra] == 7).all())
    got = out.reshape(-1, H, D)
    want, size = [], []
    for i in range(len(lens_q)):
        a, b = slice(cu_q[i], cu_q[i + 1]), slice(cu_k[i], cu_k[i + 1])
        o, s = ref.attend(q[a].reshape(-1, H, D), k[b].reshape(-1, Hkv, D), v[b].reshape(-1, Hkv, D), scale)
        want.append(o)
        size.append(s)
    want, size = torch.cat(want), torch.cat(size)
    close(got, want, BF16 * want.abs() + (BF16 + EVAL) * size + 1e-30)
    return got, want


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 2), (7, 1), (32, 8), (16, 1), (3, 3), (40, 5), (24, 2)])
def test_prefill_lengths_and_heads(H, Hkv, D):
    run_prefill([1, 77, 0, 128, 129, 300], [1, 77, 0, 128, 129, 300], H, Hkv, D)


@pytest.mark.parametrize("D,H,Hkv", [(128, 8, 2), (64, 4, 4), (128, 5, 1)])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]), ([1], [1000]), ([100, 3, 64], [500, 3, 2000]), ([256], [257]), ([255], [511]),
    ([40, 0, 7], [0, 5, 3]),            # rows that see nothing; keys without queries
    ([513], [513]), ([700, 1, 1], [130, 1, 128]),
    ([3] * 300, [5] * 300),             # more sequences than one launch takes
    ([1200], [1200])])
def test_prefill_chunks(lens_q, lens_k, D, H, Hkv):
    run_prefill(lens_q, lens_k, H, Hkv, D, extra=24)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scores_that_grow(D):
    """Later keys score far above earlier ones: the running maximum has to follow, block after block."""
    def grow(q, k, v, cu_q, cu_k):
        n = len(k)
        k.mul_(torch.linspace(0.01, 8.0, n, device="cuda")[:, None])
        q.abs_()
        k.abs_()
    run_prefill([900, 300], [900, 300], 4, 2, D, fix=grow, scale=0.2)
    # and negative ones, where nothing may come from a maximum that starts at zero
    run_prefill([300], [300], 4, 2, D, fix=lambda q, k, v, a, b: (q.abs_().add_(1), k.abs_().neg_().sub_(1)), scale=0.3)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D,H,Hkv", [(128, 4, 1), (64, 2, 2), (128, 7, 1)])
def test_prefill_bad_values_stay_where_they_are_seen(bad, D, H, Hkv):
    def plant(q, k, v, cu_q, cu_k):
        v[cu_k[1] + 200, 5] = bad       # sequence 1: seen from its token 200 on
        v[cu_k[2], 0] = bad             # first token: everybody in sequence 2
        k[cu_k[3] + 90] = math.nan      # scores of sequence 3 from token 90 on
    got, want = run_prefill([130, 333, 70, 140], [130, 333, 70, 140], H, Hkv, D, fix=plant)
    assert bool(got[:130].isfinite().all()) and bool(got[130:330].isfinite().all())
    assert not bool(got[330:463, 0, 5].isfinite().any())
    assert bool(got[533:623].isfinite().all()) and bool(got[623:].isnan().all())


@pytest.mark.parametrize("D,H,Hkv", [(128, 8, 2), (64, 4, 4), (128, 5, 1), (64, 16, 1)])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [9000]), ([1], [1409]), ([70], [3333]), ([300], [2500]), ([1, 40, 0, 9], [1500, 4000, 17, 3]),
    ([600], [600]), ([1500], [1500]), ([2000, 30], [1100, 30])])
def test_prefill_few_rows_over_many_keys(lens_q, lens_k, D, H, Hkv):
    """Few items, cut along the keys: parts of one block, parts that some row or tile does not reach."""
    run_prefill(lens_q, lens_k, H, Hkv, D, extra=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(7, 1), (14, 2), (3, 1), (12, 1), (33, 3), (100, 1), (130, 1)])
@pytest.mark.parametrize("lens_q,lens_k", [([1, 2, 0, 1], [6, 7, 3, 1]), ([5] * 40, [9] * 40), ([3], [3000]), ([35, 150], [35, 170])])
def test_prefill_heads_that_leave_slots_empty(lens_q, lens_k, H, Hkv, D):
    run_prefill(lens_q, lens_k, H, Hkv, D, extra=8)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_few_rows_values_of_far_parts(D):
    """Scores that grow from part to part, values that are not finite in the first and the last one."""
    def plant(q, k, v, cu_q, cu_k):
        k.mul_(torch.linspace(0.01, 4.0, len(k), device="cuda")[:, None])
        v[1990, 3] = math.inf   # seen from row 30 of sequence 0 on
        v[cu_k[1] + 5, 7] = math.nan
    got, _ = run_prefill([40, 20], [2000, 1800], 4, 1, D, fix=plant)
    assert bool(got[:30].isfinite().all()) and not bool(got[30:40, :, 3].isfinite().any())
    assert bool(got[40:, :, :7].isfinite().all()) and not bool(got[40:, :, 7].isfinite().any())


def test_prefill_unused_rows_may_hold_anything():
    """Rows around the sequences' own: q rows past a tile's end, k and v of the neighbours."""
    def plant(q, k, v, cu_q, cu_k):
        q[cu_q[1]:cu_q[2]] = math.nan
        k[cu_k[1]:cu_k[2]] = math.inf
        v[cu_k[1]:cu_k[2]] = math.nan
    got, _ = run_prefill([50, 60, 70], [50, 60, 70], 4, 2, 128, fix=plant)
    assert bool(got[:50].isfinite().all()) and bool(got[110:].isfinite().all()) and bool(got[50:110].isnan().all())


def test_prefill_small_and_zero_scale():
    run_prefill([200], [260], 4, 2, 128, scale=0.0)
    run_prefill([200], [260], 4, 2, 64, scale=-0.1)


def test_prefill_is_deterministic_and_runs_on_its_stream():
    g = gen(9)
    H, Hkv, D, n = 8, 2, 128, 1000
    q, k, v = rows(n, H * D, g), rows(n, Hkv * D, g), rows(n, Hkv * D, g)
    outs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (torch.cuda.current_stream(), s, s):
        o = torch.zeros(n, H * D, dtype=bf, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        abi.m2_attn_prefill_varlen(q, H * D, k, Hkv * D, v, Hkv * D, o, H * D, H, Hkv, D, [0, 400, n], [0, 400, n], 0.1, st)
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------------ single tokens over the cache

def run_decode(lens, H, Hkv, D, seed=0, spread=1.0, scale=None, fix=None, width=None, first_page=0):
    g = gen(seed + 17)
    c = Cache(lens, Hkv, D, seed, width=width, first_page=first_page)
    cu = offsets(lens)
    k, v = rows(cu[-1], Hkv * D, g), rows(cu[-1], Hkv * D, g, 0, 0.3)
    if fix:
        fix(k, v, cu)
    c.append(k, v, cu, [0] * len(lens))
    q = rows(len(lens), H * D, g, 8, spread)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = D ** -0.5 if scale is None else scale
    ws = _empty((abi.m2_attn_decode_kv4_workspace_bytes(len(lens), H, Hkv, D),), torch.uint8, "cuda")
    ws.fill_(255)
    _, out = out_rows(len(lens), H * D, 16)
    call = lambda o=out: abi.m2_attn_decode_kv4(c.struct, q, q.stride(0), o, o.stride(0), H, kv_len, scale, ws,  # noqa: E731
                                                ws.numel(), torch.cuda.current_stream())
    call()
    ks, vs = ref.rounded_rows(k.view(-1, Hkv, D)), ref.rounded_rows(v.view(-1, Hkv, D))
    want, size = [], []
    for i in range(len(lens)):
        o, s = ref.attend(q[i].reshape(1, H, D), ks[cu[i]:cu[i + 1]], vs[cu[i]:cu[i + 1]], scale)
        want.append(o)
        size.append(s)
    want, size = torch.cat(want), torch.cat(size)
    close(out.reshape(-1, H, D), want, BF16 * want.abs() + (F16 + EVAL) * size + 1e-30)
    return dict(c=c, q=q, out=out, len=kv_len, want=want, size=size, call=call, k=k, v=v, ws=ws, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(32, 8), (1, 1), (4, 4), (7, 1), (8, 1), (16, 1), (9, 1), (40, 2), (33, 1), (6, 2)])
def test_decode_lengths_and_heads(H, Hkv, D):
    run_decode([1, 63, 64, 0, 65, 128, 129, 700, 1], H, Hkv, D)


@pytest.mark.parametrize("lens,H,Hkv,D", [
    ([1], 1, 1, 64), ([20000], 8, 1, 128), ([5000, 3], 32, 8, 128), ([50] * 300, 4, 2, 64), ([0, 0], 4, 2, 128),
    ([4096] * 5, 16, 16, 64), ([1, 40000, 77, 64 * 31], 4, 1, 128), ([900] * 40, 32, 8, 128)])
def test_decode_splits(lens, H, Hkv, D):
    run_decode(lens, H, Hkv, D)


def test_decode_scores_that_grow():
    def grow(k, v, cu):
        k.abs_().mul_(torch.linspace(0.01, 4.0, len(k), device="cuda")[:, None])
    run_decode([3000, 500], 8, 2, 128, fix=grow, scale=0.3)
    run_decode([3000, 500], 8, 2, 64, fix=lambda k, v, cu: k.abs_().neg_(), scale=0.5)


@pytest.mark.parametrize("q_spread,v_spread", [(1e-3, 1e-3), (300.0, 2000.0), (1.0, 3e-5), (1e-30, 1.0)])
def test_decode_ranges(q_spread, v_spread):
    """Magnitudes far from one: the query is scaled into f16's range exactly, values keep theirs."""
    run_decode([333, 70], 8, 2, 128, spread=q_spread, scale=0.05 / max(q_spread, 0.1),
               fix=lambda k, v, cu: v.mul_(v_spread / 0.3))


def test_decode_bad_values():
    """NaN groups reach exactly the heads, sequences and channels that see them; what lies past the length does not."""
    Hkv, D, H = 2, 128, 8
    n = [100, 300, 65]

    def plant(k, v, cu):
        v[cu[1] + 299, 3] = math.nan         # sequence 1, kv head 0, channels 0..15
        k[cu[2] + 1, D + 4] = math.nan       # sequence 2, kv head 1: all scores of its heads
    r = run_decode(n, H, Hkv, D, fix=plant)
    out = r["out"].reshape(-1, H, D)
    assert bool(out[0].isfinite().all())
    assert bool(out[1, :4, :16].isnan().all()) and bool(out[1, :4, 16:].isfinite().all())
    assert bool(out[2, 4:].isnan().all()) and bool(out[2, :4].isfinite().all())
    # one token fewer: the NaN of sequence 1 lies past the length, in the same page
    r["len"].copy_(torch.tensor([100, 299, 0], dtype=torch.int32))
    r["call"]()
    out = r["out"].reshape(-1, H, D)
    assert bool(out[:2].isfinite().all()) and bool((out[2] == 0).all())


def test_decode_leaves_out_bad_pages():
    r = run_decode([200, 150, 64], 4, 2, 64, width=5)
    H, Hkv, D = 4, 2, 64
    r["c"].table[0, 1] = r["c"].n_pages
    r["c"].table[1, 0] = -1
    r["len"][2] = 64 * 5 + 1  # past the table: cut to it, and its unset pages are left out
    abi.m2_device_status(clear=True)
    r["call"]()
    assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
    ks, vs = ref.rounded_rows(r["k"].view(-1, Hkv, D)), ref.rounded_rows(r["v"].view(-1, Hkv, D))
    keep = [list(range(64)) + list(range(128, 200)), list(range(64, 150)), list(range(64))]
    cu = [0, 200, 350]
    for i in range(3):
        at = torch.tensor(keep[i], device="cuda") + cu[i]
        want, size = ref.attend(r["q"][i].reshape(1, H, D), ks[at], vs[at], r["scale"])
        close(r["out"][i].reshape(1, H, D), want, BF16 * want.abs() + (F16 + EVAL) * size + 1e-30)


def test_decode_is_deterministic():
    r = run_decode([7000, 33, 900], 8, 2, 128)
    first = r["out"].clone()
    for _ in range(5):
        r["ws"].random_(0, 255)
        r["call"]()
        assert torch.equal(r["out"], first)


def test_decode_pages_past_32_bits():
    """A pool of more than 4 GB: the sequence's pages lie at its end."""
    first = (1 << 32) // abi.m2_kv4_page_bytes(8, 128) + 10
    run_decode([300, 1000], 8, 8, 128, first_page=first)


def test_decode_replayed_while_lengths_grow():
    """A captured step (append, attention, advance) replayed: every replay sees one token more."""
    H, Hkv, D, B, start, steps = 8, 2, 128, 3, [0, 63, 190], 4
    c = Cache([s + steps + 1 for s in start], Hkv, D, 3)
    g = gen(5)
    pre = offsets(start)
    k0, v0 = rows(pre[-1], Hkv * D, g), rows(pre[-1], Hkv * D, g)
    c.append(k0, v0, pre, [0] * B)
    pos = torch.tensor(start, dtype=torch.int32, device="cuda")
    n = pos + 1
    k, v, q = (torch.zeros(B, w * D, dtype=bf, device="cuda") for w in (Hkv, Hkv, H))
    out = torch.zeros(B, H * D, dtype=bf, device="cuda")
    ws = torch.empty(abi.m2_attn_decode_kv4_workspace_bytes(B, H, Hkv, D), dtype=torch.uint8, device="cuda")

    def step(s):
        abi.m2_kv4_append(c.struct, k, Hkv * D, v, Hkv * D, [0, 1, 2, 3], pos, s)
        abi.m2_attn_decode_kv4(c.struct, q, H * D, out, H * D, H, n, 0.1, ws, ws.numel(), s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    keep, pool = c.pages.clone(), None
    with torch.cuda.stream(side):
        step(side)  # the first launches load the kernels
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    c.pages.copy_(keep)
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
        pos.add_(1)
        n.add_(1)
    ks = [[ref.rounded_rows(k0[pre[i]:pre[i + 1]].view(-1, Hkv, D))] for i in range(B)]
    vs = [[ref.rounded_rows(v0[pre[i]:pre[i + 1]].view(-1, Hkv, D))] for i in range(B)]
    for _ in range(steps):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(B):
            ks[i].append(ref.rounded_rows(k[i].view(1, Hkv, D)))
            vs[i].append(ref.rounded_rows(v[i].view(1, Hkv, D)))
            want, size = ref.attend(q[i].view(1, H, D), torch.cat(ks[i]), torch.cat(vs[i]), 0.1)
            close(out[i].view(1, H, D), want, BF16 * want.abs() + (F16 + EVAL) * size + 1e-30)
