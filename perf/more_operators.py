"""Cases of the operators that try drafted tokens on a hybrid stack and keep those that hold.

A draft model proposes a tree of tokens for every sequence: nodes 0 .. n-1 (at most 64), node 0 the
last token that is certain, parent[r] < r.  One pass of the stack runs all nodes; verification walks
the tree; then each layer keeps the accepted path.  Five operators, in the order of their use:

  scan    the causal conv and the Mamba-2 state over the tree: every node continues its parent
  attend  attention of the nodes over the paged 4-bit cache: the context and their own ancestors,
          whose rows stand behind it (node r's at token L + r)
  verify  the walk: a node is accepted or not by its own random number, its token's probability under
          the target and under the draft; then one token from what the target leaves over
  commit  the Mamba-2 state, conv ring and position moved along the accepted path
  keep    the accepted nodes' cache rows moved together (and read back, as the next chunk would)

The 4-bit cache holds, for a page of 64 tokens and one kv head (D = head_dim), 72 * D bytes:
  K codes  64 * D/2 bytes: token t's row is [c < 4][g < D/16][h < 2], low nibble of byte (c, g, h)
           channel 16g + 4c + 2h, high nibble the next one
  V codes  64 * D/2 bytes: [b < 8][r < 8][c < 4][i < D/8], low nibble channel 8i + r of token
           8b + 2c, high nibble the same channel of the next token
  K scales 64 * D/16 bytes: [t][g], one for the channels 16g .. 16g + 15 of token t
  V scales 64 * D/16 bytes: [t / 2][g / 2][t % 2][g % 2]
A code is a sign (bit 3) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte has 5 exponent and 3
mantissa bits (bias 15, e = 0: m * 2^-17).
"""
import math
import random

import torch

own = False

PAGE = 64
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    """The heads, states and widths are those of the 4096-wide layers: 32 query and 8 kv heads of 128; 128 state
    heads of 64 channels and 128 states in 8 groups, 4 taps."""
    wide = dict(heads=32, kv_heads=8, head_dim=128)
    ssm = dict(nheads=128, chans=64, states=128, groups=8, taps=4)
    return [
        # one conversation, a short chain of drafted tokens: latency
        dict(name="attend chain 5", op="attend", nseq=1, n_min=5, n_max=5, past_min=700, past_max=700, chain=True,
             **wide),
        # a serving batch, every conversation at its own length, three tokens drafted
        dict(name="attend batch 64 chains", op="attend", nseq=64, n_min=4, n_max=4, past_min=64, past_max=4096,
             chain=True, **wide),
        # fewer conversations, wider drafts
        dict(name="attend batch 16 trees", op="attend", nseq=16, n_min=9, n_max=16, past_min=100, past_max=4000,
             chain=False, **wide),
        # two long documents and the largest trees
        dict(name="attend long 64 nodes", op="attend", nseq=2, n_min=64, n_max=64, past_min=30000, past_max=30000,
             chain=False, **wide),
        # one conversation, a small vocabulary: latency
        dict(name="verify chain 5", op="verify", nseq=1, n_min=5, n_max=5, vocab=32000, chain=True, drafted="f32"),
        # the serving batch with a large vocabulary
        dict(name="verify batch 64", op="verify", nseq=64, n_min=5, n_max=8, vocab=131072, chain=False,
             drafted="f32"),
        # one conversation: latency
        dict(name="scan chain 5", op="scan", nseq=1, n_min=5, n_max=5, chain=True, **ssm),
        # a batch of trees
        dict(name="scan batch 16 trees", op="scan", nseq=16, n_min=9, n_max=16, chain=False, **ssm),
        dict(name="commit one", op="commit", nseq=1, n_min=5, n_max=5, chain=True, **ssm),
        dict(name="commit batch 64", op="commit", nseq=64, n_min=4, n_max=8, chain=False, **ssm),
        dict(name="keep one", op="keep", nseq=1, n_min=16, n_max=16, past_min=300, past_max=300, chain=False, **wide),
        dict(name="keep batch 16", op="keep", nseq=16, n_min=9, n_max=64, past_min=64, past_max=512, chain=False,
             **wide),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "verify", "scan", "commit", "keep"])
    n = _log(rng, 1, 64)
    case = dict(op=op, n_min=rng.randint(1, n), n_max=n, chain=rng.random() < 0.4)
    if op in ("attend", "keep"):
        kv = rng.choice([1, 2, 4, 8])
        case.update(heads=kv * rng.choice([1, 2, 3, 4, 7, 8] if kv < 8 else [1, 2, 4]), kv_heads=kv,
                    head_dim=rng.choice([64, 128]))
        case.update(nseq=_log(rng, 1, 64 if op == "attend" else 32))
        top = max(2, min(30000, (150000 if op == "attend" else 12000) // case["nseq"]))
        if op == "attend":
            top = max(2, min(top, 3000000 // (case["nseq"] * n)))
        a = _log(rng, 1, top)
        case.update(past_min=rng.randint(0, a), past_max=a)
    elif op == "verify":
        # no more than the listed batch's rows
        vocab = _log(rng, 100, 200000)
        case.update(vocab=vocab, nseq=_log(rng, 1, max(1, min(64, 60000000 // (vocab * n)))))
        case.update(drafted=rng.choice(["f32", "bf16", "none"]))
    else:
        heads = rng.choice([8, 40, 64, 128])
        case.update(nheads=heads, chans=rng.choice([32, 64, 128] if heads < 128 else [32, 64]),
                    states=rng.choice([16, 32, 64, 128]), groups=rng.choice([1, 2, 8]), taps=rng.choice([2, 4, 4]))
        most = 16 if op == "scan" else 64
        case.update(nseq=_log(rng, 1, max(1, min(most, 1024 // n)) if op == "scan" else most))
    return case


def _lengths(case, what):
    """The sequences' lengths: the case's own, whatever the seed; the first is the longest."""
    lo, hi = case[what + "_min"], case[what + "_max"]
    rng = random.Random("%s %d %d %d" % (what, lo, hi, case["nseq"]))
    return [hi] + [rng.randint(lo, hi) for _ in range(case["nseq"] - 1)]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _parents(case):
    """A tree a sequence, the case's own: a chain, or one in which nodes have up to a few children."""
    rng = random.Random("tree %d %d %d" % (case["n_min"], case["n_max"], case["nseq"]))
    return [[-1] + [r - 1 if case["chain"] else rng.randint((r - 1) // 2, r - 1) for r in range(1, n)]
            for n in _lengths(case, "n")]


def _depths(tree):
    d = []
    for p in tree:
        d.append(1 if p < 0 else d[p] + 1)
    return d


def work(case):
    n = _lengths(case, "n")
    if case["op"] in ("attend", "keep"):
        H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
        past, row = _lengths(case, "past"), case["kv_heads"] * case["head_dim"] * 2 * 0.5625
        if case["op"] == "attend":
            pairs = sum(a * b + sum(_depths(t)) for a, b, t in zip(n, past, _parents(case)))
            return {"bytes": (sum(n) + sum(past)) * row + 4 * D * H * sum(n), "flops": 4 * D * H * pairs}
        # half of the nodes are moved; every row is read back
        return {"bytes": sum(n) * row + (sum(n) + sum(past)) * (row + 4 * K * D), "flops": 2 * (sum(n) + sum(past)) * K * D}
    if case["op"] == "verify":
        # the row of the last accepted node, and the draft's where something was refused there
        size = 2 if case["drafted"] == "bf16" else 4
        return {"bytes": case["nseq"] * case["vocab"] * size * (1 if case["drafted"] == "none" else 2) + 28 * sum(n),
                "flops": 4 * case["nseq"] * case["vocab"]}
    H, P, N, G = case["nheads"], case["chans"], case["states"], case["groups"]
    state, width = H * P * N, H * P + 2 * G * N
    if case["op"] == "scan":
        pairs = sum(sum(_depths(t)) for t in _parents(case))
        return {"bytes": 4 * state * len(n) + 2 * (case["taps"] - 1) * width * len(n)
                + sum(n) * (4 * width + 4 * H * P + 2 * H),
                "flops": 2 * state * sum(n) + pairs * 2 * (G * N + H * P) + sum(n) * 2 * case["taps"] * width}
    kept = (sum(n) + len(n)) // 2
    return {"bytes": 8 * state * len(n) + 4 * (case["taps"] - 1) * width * len(n) + kept * 2 * (width + H),
            "flops": 4 * state * kept}


# ------------------------------------------------------------------ inputs

def _scale_bytes(amax):
    """Largest magnitudes of groups -> scale bytes and the scales, fp32."""
    t = (amax / 6.0).clamp(max=10240.0)
    e = (torch.frexp(t)[1] - 1).clamp(min=-14)
    step = torch.ldexp(torch.ones_like(t), e - 3)
    m = torch.round(t / step)  # at most 16: a carry into the next exponent
    byte = torch.where(m < 8, m.int(), ((e + 15) << 3) + (m.int() - 8))
    return byte.to(torch.uint8), (m * step)


def _codes(x, scale):
    """fp32 channels [..., 16] over their scale [..., 1] -> codes (ties to the even code)."""
    a = x.abs()
    c = ((a > 0.25 * scale).to(torch.uint8) + (a >= 0.75 * scale) + (a > 1.25 * scale) + (a >= 1.75 * scale)
         + (a > 2.5 * scale) + (a >= 3.5 * scale) + (a > 5.0 * scale))
    c = torch.where(scale > 0, c, torch.zeros_like(c))
    return (c + 8 * (x < 0) * (c > 0)).to(torch.uint8)


def _pool(n_pages, K, D, gen):
    """A pool of pages whose every slot holds quantized random keys and values."""
    def half(spread):
        x = torch.randn(n_pages, K, PAGE, D // 16, 16, device="cuda", generator=gen) * spread
        b, s = _scale_bytes(x.abs().amax(-1, keepdim=True))
        return _codes(x, s).view(n_pages, K, PAGE, D), b.view(n_pages, K, PAGE, D // 16)
    pages = torch.empty(n_pages, K, 72 * D, dtype=torch.uint8, device="cuda")
    c, s = half(1.0)
    c = c.view(n_pages, K, PAGE, D // 16, 4, 2, 2).permute(0, 1, 2, 4, 3, 5, 6)
    pages[..., :32 * D] = (c[..., 0] | (c[..., 1] << 4)).reshape(n_pages, K, 32 * D)
    pages[..., 64 * D:68 * D] = s.reshape(n_pages, K, 4 * D)
    c, s = half(0.5)
    c = c.view(n_pages, K, 8, 4, 2, D // 8, 8).permute(0, 1, 2, 6, 3, 5, 4)
    pages[..., 32 * D:64 * D] = (c[..., 0] | (c[..., 1] << 4)).reshape(n_pages, K, 32 * D)
    pages[..., 68 * D:] = s.view(n_pages, K, PAGE // 2, 2, D // 32, 2).permute(0, 1, 2, 4, 3, 5).reshape(n_pages, K, 4 * D)
    return pages


def _table(lens, rng):
    """Pages for `lens` tokens a sequence, in any order: (table rows, pages in the pool)."""
    need = [-(-n // PAGE) for n in lens]
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    width = max(1, max(need))
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), len(ids)


def _paths(trees, rng):
    """An accepted path a tree: from node 0 to a random node."""
    flat, counts = [], []
    for t in trees:
        path, r = [], rng.randrange(len(t))
        while r >= 0:
            path.append(r)
            r = t[r]
        flat += path[::-1] + [-1] * (len(t) - len(path))
        counts.append(len(path))
    return flat, counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    bf = torch.bfloat16
    s = dict(case)
    n, trees = _lengths(case, "n"), _parents(case)
    s["cu"], T = _offsets(n), sum(n)
    s["parent"] = ints([p for t in trees for p in t])
    if case["op"] in ("commit", "keep"):
        path, count = _paths(trees, rng)
        s["path"], s["count"] = ints(path), ints(count)
    if case["op"] in ("attend", "keep"):
        H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
        past = _lengths(case, "past")
        lens = [a + b for a, b in zip(n, past)]
        s["table"], n_pages = _table(lens, rng)
        s["pages"] = _pool(n_pages, K, D, gen)
        s["past"], s["cu_all"] = ints(past), _offsets(lens)
        if case["op"] == "attend":
            s["q"] = randn(T, H * D).to(bf)
            s["out"] = torch.empty(T, H * D, dtype=bf, device="cuda")
            s["ws"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # a program's scratch, for all its calls
        else:
            s["k_out"] = torch.empty(sum(lens), K * D, dtype=bf, device="cuda")
            s["v_out"] = torch.empty(sum(lens), K * D, dtype=bf, device="cuda")
    elif case["op"] == "verify":
        # a draft that mostly agrees with the target; siblings are drawn from one row
        V = case["vocab"]
        p, size = 2.5 * randn(T, V), torch.bfloat16 if case["drafted"] == "bf16" else torch.float32
        q = torch.softmax(p + 0.7 * randn(T, V), -1)
        p = torch.softmax(p, -1)
        above = (s["parent"].long().clamp(min=0)
                 + torch.tensor([c for c, k in zip(s["cu"], n) for _ in range(k)], device="cuda"))
        # the place in the draft's cumulated row where a random number falls
        total = torch.cumsum(q, -1)
        at = torch.rand(T, 1, device="cuda", generator=gen) * total[above, -1:]
        s["token"] = torch.searchsorted(total[above], at)[:, 0].clamp(max=V - 1).int()
        s["p"], s["q"] = p.to(size), None if case["drafted"] == "none" else q.to(size)
        s["u"] = torch.rand(T, device="cuda", generator=gen)
        s["u_next"] = torch.rand(case["nseq"], device="cuda", generator=gen)
        s["path"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["count"] = torch.empty(case["nseq"], dtype=torch.int32, device="cuda")
        s["next"] = torch.empty(case["nseq"], dtype=torch.int32, device="cuda")
    else:
        H, P, N, G, B = case["nheads"], case["chans"], case["states"], case["groups"], case["nseq"]
        width, ring = H * P + 2 * G * N, case["taps"] - 1
        s["width"] = width
        # rows of the input projection: z, x | B | C, dt (padded to 8)
        s["ld"] = (H * P + width + H + 7) // 8 * 8
        s["zx"] = randn(T, s["ld"]).to(bf)
        s["h"], s["ring"] = 0.3 * randn(B, H, P, N), randn(B, ring, width).to(bf)
        s["pos"] = ints([rng.randint(0, 5000) for _ in range(B)])
        s["conv_w"], s["conv_b"] = (0.5 * randn(width, case["taps"])).to(bf), (0.1 * randn(width)).to(bf)
        s["A_log"] = torch.rand(H, device="cuda", generator=gen) * math.log(16.0)
        s["D"] = 1 + 0.1 * randn(H)
        dt0 = torch.exp(torch.rand(H, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
        if case["op"] == "scan":
            s["u"] = torch.empty(T, width, dtype=bf, device="cuda")
            s["y"] = torch.empty(T, H * P, device="cuda")
        else:
            s["u"] = torch.nn.functional.silu(randn(T, width)).to(bf)
            s["h_out"], s["ring_out"] = torch.empty_like(s["h"]), torch.empty_like(s["ring"])
            s["pos_out"] = torch.empty_like(s["pos"])
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from mamba_ssm_layer_gb300 import abi

    stream = torch.cuda.current_stream()
    if s["op"] in ("attend", "keep"):
        H, K, D = s["heads"], s["kv_heads"], s["head_dim"]
        cache = abi.kv4_cache(s["pages"], s["pages"].shape[0], K, D, s["table"], s["nseq"], s["table"].shape[1])
        if s["op"] == "attend":
            abi.m2_attn_tree_kv4(cache, s["q"], H * D, s["out"], H * D, H, s["cu"], s["parent"], s["past"], D ** -0.5,
                                 s["ws"], s["ws"].numel(), stream)
            return s["out"]
        abi.m2_kv4_keep(cache, s["cu"], s["path"], s["count"], s["past"], stream)
        abi.m2_kv4_gather(cache, s["k_out"], K * D, s["v_out"], K * D, s["cu_all"], stream)
        return s["k_out"], s["v_out"]
    if s["op"] == "verify":
        fmt = abi.M2_PROB_BF16 if s["drafted"] == "bf16" else abi.M2_PROB_F32
        abi.m2_verify_tree(s["p"], s["vocab"], s["q"], s["vocab"], fmt, s["vocab"], s["cu"], s["parent"], s["token"],
                           s["u"], s["u_next"], s["path"], s["count"], s["next"], stream)
        return s["path"], s["count"], s["next"]
    H, P, N, G, W = s["nheads"], s["chans"], s["states"], s["groups"], s["width"]
    xbc, dt = s["zx"][:, H * P:], s["zx"][:, H * P + W:]
    if s["op"] == "scan":
        u = s["u"]
        abi.mamba2_tree_conv(s["ring"], s["pos"], xbc, s["ld"], s["conv_w"], s["conv_b"], u, W, s["cu"], s["parent"], W,
                             s["taps"], 1, stream)
        abi.mamba2_tree_ssm(s["h"], u, u[:, H * P:], u[:, H * P + G * N:], W, dt, s["ld"], s["A_log"], s["D"],
                            s["dt_bias"], s["y"], s["cu"], s["parent"], H, P, N, G, stream)
        return u, s["y"]
    abi.mamba2_tree_commit(s["h"], s["ring"], s["pos"], s["h_out"], s["ring_out"], s["pos_out"], xbc, s["ld"], s["u"],
                           W, dt, s["ld"], s["A_log"], s["dt_bias"], s["cu"], s["path"], s["count"], H, P, N, G,
                           s["taps"], stream)
    return s["h_out"], s["ring_out"], s["pos_out"]


# ------------------------------------------------------------------ the plain forms

def _padded(s):
    """Node numbers, rows and parents, padded to the largest tree: [n][m]."""
    dev = s["parent"].device
    cu = torch.tensor(s["cu"], device=dev)
    m = max(b - a for a, b in zip(s["cu"], s["cu"][1:]))
    r = torch.arange(m, device=dev)
    real = r < (cu[1:] - cu[:-1])[:, None]
    row = torch.where(real, cu[:-1, None] + r, torch.zeros_like(r))
    return m, real, row, torch.where(real, s["parent"].long()[row], -torch.ones_like(r))


def _ancestors(parent):
    """[n][m][m]: whether node j is node r or stands above it."""
    m = parent.shape[1]
    eye = torch.eye(m, device=parent.device)
    above = eye + (parent[..., None] == torch.arange(m, device=parent.device)).float()
    for _ in range(6):  # 2^6 generations
        above = (torch.matmul(above, above) > 0).float()
    return above > 0


def _value(codes):
    level = torch.tensor(LEVELS, device=codes.device)
    return level[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3))


def _scale_value(b):
    e, m = (b >> 3).int(), (b & 7).float()
    one = torch.ones_like(m)
    return torch.where(e > 0, torch.ldexp(8 * one + m, e - 18), torch.ldexp(m, torch.full_like(e, -17)))


def _unpack(pages, K, D):
    """The pool's keys and values, fp32 [pages][kv head][64][D]."""
    n = pages.shape[0]
    b = pages[..., :32 * D].reshape(n, K, PAGE, 4, D // 16, 2)
    k = torch.stack([b & 15, b >> 4], -1).permute(0, 1, 2, 4, 3, 5, 6).reshape(n, K, PAGE, D)
    b = pages[..., 32 * D:64 * D].reshape(n, K, 8, 8, 4, D // 8)
    v = torch.stack([b & 15, b >> 4], -1).permute(0, 1, 2, 4, 6, 5, 3).reshape(n, K, PAGE, D)
    ks = pages[..., 64 * D:68 * D].reshape(n, K, PAGE, D // 16)
    vs = pages[..., 68 * D:].reshape(n, K, PAGE // 2, D // 32, 2, 2).permute(0, 1, 2, 4, 3, 5)
    vs = vs.reshape(n, K, PAGE, D // 16)
    return (_value(k) * _scale_value(ks).repeat_interleave(16, -1),
            _value(v) * _scale_value(vs).repeat_interleave(16, -1))


def _attend_plain(s):
    H, K, D, n = s["heads"], s["kv_heads"], s["head_dim"], s["nseq"]
    m, real, row, parent = _padded(s)
    k, v = _unpack(s["pages"], K, D)
    page = s["table"].long().clamp(min=0)
    width = page.shape[1] * PAGE
    k = k[page].transpose(1, 2).reshape(n, K, width, D)
    v = v[page].transpose(1, 2).reshape(n, K, width, D)
    # token t is node t - past; everything before is seen
    node = torch.arange(width, device=k.device) - s["past"].long()[:, None]
    seen = (node < 0)[:, None] | (_ancestors(parent).gather(2, node.clamp(0, m - 1)[:, None].expand(n, m, width))
                                  & (node < m)[:, None])
    q = (s["q"][row].view(n, m, K, H // K, D).permute(0, 2, 1, 3, 4).float() * D ** -0.5).reshape(n, K, -1, D)
    p = torch.matmul(q, k.transpose(-1, -2))
    p.masked_fill_(~seen.repeat_interleave(H // K, 1)[:, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.view(n, K, m, H // K, D).permute(0, 2, 1, 3, 4).reshape(n, m, H * D).to(torch.bfloat16)[real]


def _keep_plain(s):
    K, D = s["kv_heads"], s["head_dim"]
    m, real, row, _ = _padded(s)
    count = s["count"].long()[:, None]
    r = torch.arange(m, device=row.device)
    seq, j = torch.nonzero(r < count, as_tuple=True)  # path entry j of a sequence
    past = s["past"].long()[seq]
    at, to = past + s["path"].long()[row][seq, j], past + j

    def move(lo, hi, size, pair):
        """Codes or scales [pages][K][64][size], one a byte, moved and put back."""
        flat = s["pages"][..., lo:hi]
        x = pair(flat)
        table = s["table"].long()
        x[table[seq, to // PAGE], :, to % PAGE] = x[table[seq, at // PAGE], :, at % PAGE]
        return x

    def v_codes(b):
        b = b.reshape(-1, K, 8, 8, 4, D // 8)
        return torch.stack([b & 15, b >> 4], -1).permute(0, 1, 2, 4, 6, 5, 3).reshape(-1, K, PAGE, D)

    def v_scales(b):
        b = b.reshape(-1, K, PAGE // 2, D // 32, 2, 2)
        return b.permute(0, 1, 2, 4, 3, 5).reshape(-1, K, PAGE, D // 16)

    pages = s["pages"]
    kc = move(0, 32 * D, D // 2, lambda b: b.reshape(-1, K, PAGE, D // 2).clone())
    vc = move(32 * D, 64 * D, D, v_codes)
    ks = move(64 * D, 68 * D, D // 16, lambda b: b.reshape(-1, K, PAGE, D // 16).clone())
    vs = move(68 * D, 72 * D, D // 16, v_scales)
    pages[..., :32 * D] = kc.reshape(-1, K, 32 * D)
    c = vc.view(-1, K, 8, 4, 2, D // 8, 8).permute(0, 1, 2, 6, 3, 5, 4)
    pages[..., 32 * D:64 * D] = (c[..., 0] | (c[..., 1] << 4)).reshape(-1, K, 32 * D)
    pages[..., 64 * D:68 * D] = ks.reshape(-1, K, 4 * D)
    pages[..., 68 * D:] = vs.view(-1, K, PAGE // 2, 2, D // 32, 2).permute(0, 1, 2, 4, 3, 5).reshape(-1, K, 4 * D)
    # read back
    k, v = _unpack(pages, K, D)
    total = s["cu_all"][-1]
    cu = torch.tensor(s["cu_all"], device=k.device)
    seq = torch.repeat_interleave(torch.arange(s["nseq"], device=k.device), cu[1:] - cu[:-1], output_size=total)
    at = torch.arange(total, device=k.device) - cu[seq]
    page = s["table"].long()[seq, at // PAGE]
    return tuple(x[page, :, at % PAGE].reshape(total, K * D).to(torch.bfloat16) for x in (k, v))


def _verify_plain(s):
    """In 64 bits: cumulated probabilities are compared with random numbers."""
    m, real, row, parent = _padded(s)
    dev, n = row.device, s["nseq"]
    f = torch.float64
    seq = torch.arange(n, device=dev)
    token = s["token"].long()[row]
    cur = torch.zeros(n, dtype=torch.long, device=dev)
    took, c, total = real[:, :1].clone(), torch.zeros(n, dtype=f, device=dev), torch.ones(n, dtype=f, device=dev)
    drafted = s["q"] is not None

    def left(cur, c, gone):
        """What remains of the target's row."""
        p = s["p"][row[seq, cur]].to(f)
        if drafted:
            return (p - c[:, None] * s["q"][row[seq, cur]].to(f)).clamp_(min=0)
        return p.masked_fill_(gone, 0.0)
    gone = torch.zeros(n, s["vocab"], dtype=torch.bool, device=dev)
    for r in range(1, m):  # children stand behind their parents, siblings in order
        here = real[:, r] & (parent[:, r] == cur)
        x, at = token[:, r], row[seq, cur]
        p = s["p"][at, x].to(f)
        if drafted:
            q = s["q"][at, x].to(f)
            ok = here & (s["u"][row[:, r]].to(f) * q * total < (p - c * q).clamp(min=0))
        else:
            ok = here & (s["u"][row[:, r]].to(f) * total < torch.where(gone[seq, x], torch.zeros_like(p), p))
        took = torch.cat([took, ok[:, None]], 1)
        no = here & ~ok
        gone[seq, x] |= no
        gone &= ~ok[:, None]
        cur = torch.where(ok, r, cur)
        c = torch.where(ok, torch.zeros_like(c), torch.where(no, c + total, c))
        total = torch.where(ok, torch.ones_like(c), torch.where(no, left(cur, c, gone).sum(-1), total))
    rest = left(cur, c, gone)
    none = rest.sum(-1) <= 0
    rest = torch.where(none[:, None], s["p"][row[seq, cur]].to(f), rest).cumsum(-1)
    last = torch.searchsorted(rest, (s["u_next"].to(f) * rest[:, -1])[:, None], right=True)[:, 0]
    # accepted nodes, in order, then -1
    order = torch.where(took, torch.arange(m, device=dev), m).sort(-1)[0]
    return (torch.where(order < m, order, -1)[real].int(), took.sum(-1).int(), last.clamp(max=s["vocab"] - 1).int())


def _dt(s, rows):
    """Steps and log decays of rows [..., H]."""
    H, P = s["nheads"], s["chans"]
    v = s["zx"][rows][..., H * P + s["width"]:H * P + s["width"] + H].float() + s["dt_bias"]
    dt = torch.where(v > 20, v, torch.log1p(torch.exp(v))).clamp(1e-9, 1e9)
    return dt, -dt * torch.exp(s["A_log"])


def _scan_plain(s):
    H, P, N, G, W, L = s["nheads"], s["chans"], s["states"], s["groups"], s["width"], s["taps"] - 1
    m, real, row, parent = _padded(s)
    dev, n = row.device, s["nseq"]
    seq = torch.arange(n, device=dev)[:, None]
    # the conv: a node's row, its ancestors', then the ring from the newest token back
    x = s["zx"][row][..., H * P:H * P + W].float()
    w = s["conv_w"].float()
    at, back, taps = torch.arange(m, device=dev).expand(n, m), torch.zeros_like(parent), []
    for _ in range(L + 1):
        old = s["ring"][seq, (s["pos"].long()[:, None] - back) % L].float()
        taps.append(torch.where((at >= 0)[..., None], x[seq, at.clamp(min=0)], old))
        up = parent.gather(1, at.clamp(min=0))
        at, back = torch.where(at >= 0, up, at), torch.where((at >= 0) & (up >= 0), back, back + 1)
    v = s["conv_b"].float()
    for j in range(L + 1):  # oldest first
        v = v + taps[L - j] * w[:, j]
    u = (v / (1 + torch.exp(-v))).to(torch.bfloat16)
    f = u.float()
    X = f[..., :H * P].view(n, m, H, P)
    B = f[..., H * P:H * P + G * N].view(n, m, G, N)
    C = f[..., H * P + G * N:].view(n, m, G, N)
    dt, la = _dt(s, row)
    anc = _ancestors(parent)
    total = torch.matmul(anc.double(), la.double()).permute(0, 2, 1)  # [n][H][m]: log decay along the path
    decay = torch.where(anc[:, None], torch.exp(total[..., :, None] - total[..., None, :]).float(), 0.0)
    cb = torch.matmul(C.transpose(1, 2), B.permute(0, 2, 3, 1)).repeat_interleave(H // G, 1)  # [n][H][m][m]
    y = torch.matmul(decay * cb * dt.permute(0, 2, 1)[:, :, None], X.transpose(1, 2))
    start = torch.matmul(C.transpose(1, 2).repeat_interleave(H // G, 1), s["h"].transpose(-1, -2))
    y = y + torch.exp(total).float()[..., None] * start + s["D"][:, None, None] * X.transpose(1, 2)
    return u[real], y.transpose(1, 2).reshape(n, m, H * P)[real]


def _commit_plain(s):
    H, P, N, G, W, L = s["nheads"], s["chans"], s["states"], s["groups"], s["width"], s["taps"] - 1
    m, real, row, _ = _padded(s)
    dev, n = row.device, s["nseq"]
    first = torch.tensor(s["cu"][:-1], device=dev)
    rows = first[:, None] + s["path"].long()[row].clamp(min=0)
    count = s["count"].long()
    h, ring = s["h"].clone(), s["ring"].clone()
    seq = torch.arange(n, device=dev)
    for j in range(m):
        at, on = rows[:, j], j < count
        f = s["u"][at].float()
        x, B = f[:, :H * P].view(n, H, P), f[:, H * P:H * P + G * N].view(n, G, N).repeat_interleave(H // G, 1)
        dt, la = _dt(s, at)
        new = torch.exp(la)[..., None, None] * h + (dt[..., None] * x)[..., None] * B[:, :, None]
        h = torch.where(on[:, None, None, None], new, h)
        slot = (s["pos"].long() + j) % L
        ring[seq, slot] = torch.where(on[:, None], s["zx"][at, H * P:H * P + W], ring[seq, slot])
    return h, ring, s["pos"] + s["count"]


def run(state):
    if own:
        return _run_own(state)
    plain = {"attend": _attend_plain, "keep": _keep_plain, "verify": _verify_plain, "scan": _scan_plain,
             "commit": _commit_plain}
    return plain[state["op"]](state)


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_rows(s, seq, count):
    """The first `count` tokens of a sequence in the cache, by the position of every nibble: fp64 [K][count][D] x 2."""
    K, D = s["kv_heads"], s["head_dim"]
    dev = s["pages"].device
    tok = torch.arange(count, device=dev)
    page = s["table"][seq].long()[tok // PAGE]
    t, d, h = (tok % PAGE)[None, :, None], torch.arange(D, device=dev)[None, None], torch.arange(K, device=dev)[:, None, None]
    flat = s["pages"].view(-1)
    base = (page[None, :, None] * K + h) * 72 * D
    kb = flat[base + t * (D // 2) + (d % 16) // 4 * (D // 8) + d // 16 * 2 + d % 4 // 2]
    vb = flat[base + 32 * D + t // 8 * (4 * D) + d % 8 * (D // 2) + t % 8 // 2 * (D // 8) + d // 8]
    kb = (kb >> (4 * (d % 2)).to(torch.uint8)) & 15
    vb = (vb >> (4 * (t % 2)).to(torch.uint8)) & 15
    ksb = flat[base + 64 * D + t * (D // 16) + d // 16]
    vsb = flat[base + 68 * D + t // 2 * (D // 8) + d // 32 * 4 + t % 2 * 2 + d // 16 % 2]
    value = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=dev)
    scale = torch.tensor([(8 + b % 8) * 2.0 ** (b // 8 - 18) if b > 7 else b * 2.0 ** -17 for b in range(256)],
                         dtype=torch.float64, device=dev)
    return value[kb.long()] * scale[ksb.long()], value[vb.long()] * scale[vsb.long()]


def _exact_verify(s):
    """The walk with every remainder normalised, as the method is usually stated."""
    paths, counts, tokens = [], [], []
    parent, token = s["parent"].tolist(), s["token"].tolist()
    u, u_next = s["u"].tolist(), s["u_next"].tolist()
    for i in range(s["nseq"]):
        a, b = s["cu"][i], s["cu"][i + 1]
        path, dist = [0], s["p"][a].double()
        for r in range(1, b - a):
            if parent[a + r] != path[-1]:
                continue
            x, q = token[a + r], None if s["q"] is None else s["q"][a + path[-1]].double()
            ask = 1.0 if q is None else float(q[x])
            if u[a + r] * ask < float(dist[x]):
                path.append(r)
                dist = s["p"][a + r].double()
                continue
            if q is None:
                dist = dist.clone()
                dist[x] = 0.0
            else:
                dist = (dist - q).clamp(min=0)
            if float(dist.sum()) > 0:
                dist = dist / dist.sum()
        if float(dist.sum()) <= 0:
            dist = s["p"][a + path[-1]].double()
        run = dist.cumsum(0)
        tokens.append(int((run <= u_next[i] * run[-1]).sum().clamp(max=s["vocab"] - 1)))
        counts.append(len(path))
        paths += path + [-1] * (b - a - len(path))
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (paths, counts, tokens))


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if s["op"] == "verify":
        return _exact_verify(s)
    if s["op"] in ("attend", "keep"):
        H, K, D = s["heads"], s["kv_heads"], s["head_dim"]
        past, path, count = s["past"].tolist(), None, None
        found = [], []
        for i in range(s["nseq"]):
            a, b = s["cu"][i], s["cu"][i + 1]
            k, v = _exact_rows(s, i, past[i] + b - a)
            if s["op"] == "keep":
                order = list(range(past[i] + b - a))
                for j, r in enumerate(s["path"][a:a + int(s["count"][i])].tolist()):
                    order[past[i] + j] = past[i] + r
                for x, y in zip(found, (k, v)):
                    x.append(y[:, order].transpose(0, 1).reshape(len(order), K * D))
                continue
            parent = s["parent"][a:b].tolist()
            for r0 in range(0, b - a, 8):  # a few nodes at a time
                nodes, see = range(r0, min(b - a, r0 + 8)), []
                for r in nodes:
                    line = []
                    while r >= 0:
                        line.append(past[i] + r)
                        r = parent[r]
                    see.append(line)
                mask = torch.zeros(len(see), k.shape[1], dtype=torch.bool, device="cuda")
                mask[:, :past[i]] = True
                for m, line in zip(mask, see):
                    m[line] = True
                q = s["q"][a + r0:a + r0 + len(see)].to(f).view(-1, K, H // K, D)
                score = torch.einsum("rkgd,ktd->rkgt", q, k) / math.sqrt(D)
                prob = torch.softmax(score.masked_fill(~mask[:, None, None], -math.inf), -1)
                found[0].append(torch.einsum("rkgt,ktd->rkgd", prob, v).reshape(len(see), H * D))
        return torch.cat(found[0]) if s["op"] == "attend" else tuple(torch.cat(x) for x in found)
    H, P, N, G, W, L = s["nheads"], s["chans"], s["states"], s["groups"], s["width"], s["taps"] - 1
    if H * P * N * max(_lengths(case, "n")) > 80e6:
        return None
    z = s["zx"].to(f)
    dt = torch.nn.functional.softplus(z[:, H * P + W:H * P + W + H] + s["dt_bias"].to(f)).clamp(1e-9, 1e9)
    keep = torch.exp(-dt * torch.exp(s["A_log"].to(f)))
    group = torch.arange(H, device="cuda") // (H // G)

    def step(h, u, t):
        x, B = u[:H * P].view(H, P, 1), u[H * P:H * P + G * N].view(G, 1, N)[group]
        return keep[t].view(H, 1, 1) * h + dt[t].view(H, 1, 1) * x * B
    if s["op"] == "commit":
        hs, ring, pos = [], s["ring"].to(f), s["pos"].tolist()
        for i in range(s["nseq"]):
            h = s["h"][i].to(f)
            for j, r in enumerate(s["path"][s["cu"][i]:s["cu"][i] + int(s["count"][i])].tolist()):
                h = step(h, s["u"][s["cu"][i] + r].to(f), s["cu"][i] + r)
                ring[i, (pos[i] + j) % L] = z[s["cu"][i] + r, H * P:H * P + W]
            hs.append(h)
        return torch.stack(hs), ring, s["pos"] + s["count"]
    us, ys, pos = [], [], s["pos"].tolist()
    for i in range(s["nseq"]):
        a, b = s["cu"][i], s["cu"][i + 1]
        parent, states = s["parent"][a:b].tolist(), []
        for r in range(b - a):
            line, up = [], r
            while up >= 0 and len(line) <= L:
                line.append(z[a + up, H * P:H * P + W])
                up = parent[up]
            line += [s["ring"][i, (pos[i] - 1 - k) % L].to(f) for k in range(L + 1 - len(line))]
            v = s["conv_b"].to(f) + sum(line[L - j] * s["conv_w"][:, j].to(f) for j in range(L + 1))
            us.append(v * torch.sigmoid(v))
            # the state takes the conv's output as it is held: rounded once
            u = us[-1].to(torch.bfloat16).to(f)
            h = step(s["h"][i].to(f) if parent[r] < 0 else states[parent[r]], u, a + r)
            states.append(h)
            C = u[H * P + G * N:].view(G, 1, N)[group]
            ys.append(((h * C).sum(-1) + s["D"].to(f)[:, None] * u[:H * P].view(H, P)).reshape(-1))
    return torch.stack(us), torch.stack(ys)
