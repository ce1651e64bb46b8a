"""Cases of the attention operators that stand beside the Mamba-2 layers of a hybrid stack.

Four operators, in the order in which a layer calls them:

  rope     RMS norm of every query and key head and the rotation by position, in one pass
  cache    new key and value rows appended to a paged 4-bit cache, and the sequences read back as
           bf16 rows (what a chunked prompt attends to)
  prompt   causal attention of packed sequences of different lengths, grouped heads; a sequence's
           queries are the last rows of its keys (the whole prompt, or a chunk after cached tokens)
  step     attention of one query token a sequence over the paged 4-bit cache

The 4-bit cache holds, for a page of 64 tokens and one kv head (D = head_dim), 72 * D bytes:
  K codes  64 * D/2 bytes: token t's row is [c < 4][g < D/16][h < 2], low nibble of byte (c, g, h)
           channel 16g + 4c + 2h, high nibble the next one
  V codes  64 * D/2 bytes: [b < 8][r < 8][c < 4][i < D/8], low nibble channel 8i + r of token
           8b + 2c, high nibble the same channel of the next token
  K scales 64 * D/16 bytes: [t][g], one for the channels 16g .. 16g + 15 of token t
  V scales 64 * D/16 bytes: [t / 2][g / 2][t % 2][g % 2]
A code is a sign (bit 3) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte has 5 exponent and 3
mantissa bits (bias 15, e = 0: m * 2^-17).  A group's scale is its largest magnitude / 6, rounded to
nearest even and at most 10240; its codes are the channels over the scale, rounded to nearest even.
"""
import math
import random

import torch

own = False

PAGE = 64
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    """The heads are those of a 4096-wide layer: 32 query and 8 kv heads of 128."""
    wide = dict(heads=32, kv_heads=8, head_dim=128)
    return [
        # one decode step of 64 sequences, each somewhere in its own text
        dict(name="rope step 64", op="rope", rows=64, far=100000, norm=True, rot=128, pairs="half", **wide),
        # all rows of a long prompt
        dict(name="rope prompt 8k", op="rope", rows=8192, far=8192, norm=True, rot=128, pairs="half", **wide),
        # 16 sequences' first prompts, the lengths of the eight-layer stack's batch
        dict(name="cache prompts 16", op="cache", nseq=16, new_min=64, new_max=512, past_min=0, past_max=0, **wide),
        # the next chunk of four long conversations
        dict(name="cache chunks 4", op="cache", nseq=4, new_min=500, new_max=2048, past_min=1000, past_max=12000,
             **wide),
        # a short question, alone: latency
        dict(name="prompt short", op="prompt", nseq=1, q_min=77, q_max=77, past_min=0, past_max=0, **wide),
        # the stack's batch of 16 prompts in one call
        dict(name="prompt packed 16", op="prompt", nseq=16, q_min=64, q_max=512, past_min=0, past_max=0, **wide),
        # chunks of four conversations over what was said before, smaller heads
        dict(name="prompt chunks 4", op="prompt", nseq=4, q_min=200, q_max=1000, past_min=1000, past_max=6000,
             heads=32, kv_heads=8, head_dim=64),
        # one long document
        dict(name="prompt 8k", op="prompt", nseq=1, q_min=8192, q_max=8192, past_min=0, past_max=0, **wide),
        # one conversation, one token: latency
        dict(name="step one", op="step", nseq=1, len_min=700, len_max=700, **wide),
        # a serving batch, every conversation at its own length
        dict(name="step batch 64", op="step", nseq=64, len_min=64, len_max=4096, **wide),
        # smaller heads, every query head with its own kv head
        dict(name="step batch 16 d64", op="step", nseq=16, len_min=100, len_max=3000, heads=16, kv_heads=16,
             head_dim=64),
        # one very long document, one token
        dict(name="step 128k", op="step", nseq=1, len_min=131000, len_max=131000, **wide),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "prompt", "step"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, heads=kv * rng.choice([1, 2, 3, 4, 7, 8] if kv < 8 else [1, 2, 4]), kv_heads=kv, head_dim=dim)
    if op == "rope":
        rot = rng.choice([dim, dim // 2, 0])
        case.update(rows=_log(rng, 1, 8192), far=_log(rng, 100, 1000000), norm=rng.random() < 0.75 or rot == 0,
                    rot=rot, pairs=rng.choice(["half", "next"]))
        return case
    n = _log(rng, 1, 64)
    case.update(nseq=n)
    if op == "cache":
        top = max(2, 16000 // n)
        a, p = _log(rng, 1, top), rng.choice([0, _log(rng, 1, top)])
        case.update(new_min=rng.randint(1, a), new_max=a, past_min=rng.randint(0, p), past_max=p)
    elif op == "prompt":
        top = max(2, 4500 // n)
        a, p = _log(rng, 1, top), rng.choice([0, _log(rng, 1, top)])
        case.update(q_min=rng.randint(0, a - 1), q_max=a, past_min=rng.randint(0, p), past_max=p)
    else:
        a = _log(rng, 2, max(64, 100000 // n))
        case.update(len_min=rng.randint(1, a), len_max=a)
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


def work(case):
    H, K, D = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        n = case["rows"] * (H + K) * D
        return {"bytes": 4 * n + 4 * case["rows"], "flops": 10 * n}
    if case["op"] == "cache":
        new, past = sum(_lengths(case, "new")), sum(_lengths(case, "past"))
        row = K * D  # one of K and V
        # new rows in, their codes and scales out; all tokens' codes and scales in, their rows out
        return {"bytes": new * row * 2 * (2 + 0.5625) + past * row * 2 * 0.5625 + (new + past) * row * 2 * 2,
                "flops": 8 * (new + past) * row}
    if case["op"] == "prompt":
        q, past = _lengths(case, "q"), _lengths(case, "past")
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(q, past))
        return {"bytes": 2 * D * (2 * H * sum(q) + 2 * K * (sum(q) + sum(past))), "flops": 4 * D * H * pairs}
    n = _lengths(case, "len")
    return {"bytes": sum(n) * K * D * 2 * 0.5625 + 4 * D * H * len(n), "flops": 4 * D * H * sum(n)}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    H, K, D = case["heads"], case["kv_heads"], case["head_dim"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(torch.bfloat16)

    s = dict(case)
    if case["op"] == "rope":
        T, rot = case["rows"], case["rot"]
        s["qkv"] = randn(T, (H + 2 * K) * D)  # rows of the projection: queries, keys, values
        s["q_w"] = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen)).to(torch.bfloat16) if case["norm"] else None
        s["k_w"] = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen)).to(torch.bfloat16) if case["norm"] else None
        if T == case["far"]:
            s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32)
        else:
            s["pos"] = torch.randint(0, case["far"], (T,), device="cuda", generator=gen, dtype=torch.int32)
        s["theta"] = 10000.0
        # turns a position, in units of 2^-64
        s["steps"] = torch.tensor([int(2.0 ** 64 * s["theta"] ** (-2.0 * i / rot) / (2 * math.pi))
                                   for i in range(rot // 2)], dtype=torch.int64, device="cuda") if rot else None
        s["q_out"] = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(T, K * D, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "cache":
        new, past = _lengths(case, "new"), _lengths(case, "past")
        lens = [a + b for a, b in zip(new, past)]
        s["cu_new"], s["cu_all"] = _offsets(new), _offsets(lens)
        s["table"], n_pages = _table(lens, rng)
        s["pages"] = _pool(n_pages, K, D, gen)
        s["past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        s["kv"] = randn(sum(new), 2 * K * D)  # keys, values
        s["k_out"] = torch.empty(sum(lens), K * D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(sum(lens), K * D, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "prompt":
        q, past = _lengths(case, "q"), _lengths(case, "past")
        s["cu_q"], s["cu_k"] = _offsets(q), _offsets([a + b for a, b in zip(q, past)])
        s["q"] = randn(s["cu_q"][-1], H * D)
        s["k"] = randn(s["cu_k"][-1], K * D)
        s["v"] = randn(s["cu_k"][-1], 2 * K * D)[:, K * D:]  # a part of wider rows
        s["out"] = torch.empty(s["cu_q"][-1], H * D, dtype=torch.bfloat16, device="cuda")
    else:
        lens = _lengths(case, "len")
        s["table"], n_pages = _table(lens, rng)
        s["pages"] = _pool(n_pages, K, D, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = randn(len(lens), H * D)
        s["out"] = torch.empty(len(lens), H * D, dtype=torch.bfloat16, device="cuda")
        s["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # a program's scratch, for all its calls
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from mamba_ssm_layer_gb300 import abi

    H, K, D = s["heads"], s["kv_heads"], s["head_dim"]
    stream = torch.cuda.current_stream()
    if s["op"] == "rope":
        qkv, w = s["qkv"], (H + 2 * K) * D
        abi.m2_qk_norm_rope(qkv, w, qkv[:, H * D:], w, s["q_out"], H * D, s["k_out"], K * D, s["q_w"], s["k_w"],
                            s["pos"], s["steps"], s["rows"], H, K, D, s["rot"], s["pairs"] == "next", EPS, stream)
        return s["q_out"], s["k_out"]
    if s["op"] == "cache":
        cache = abi.kv4_cache(s["pages"], s["pages"].shape[0], K, D, s["table"], s["nseq"], s["table"].shape[1])
        kv = s["kv"]
        abi.m2_kv4_append(cache, kv, 2 * K * D, kv[:, K * D:], 2 * K * D, s["cu_new"], s["past"], stream)
        abi.m2_kv4_gather(cache, s["k_out"], K * D, s["v_out"], K * D, s["cu_all"], stream)
        return s["k_out"], s["v_out"]
    if s["op"] == "prompt":
        abi.m2_attn_prefill_varlen(s["q"], H * D, s["k"], K * D, s["v"], 2 * K * D, s["out"], H * D, H, K, D,
                                   s["cu_q"], s["cu_k"], D ** -0.5, stream)
        return s["out"]
    cache = abi.kv4_cache(s["pages"], s["pages"].shape[0], K, D, s["table"], s["nseq"], s["table"].shape[1])
    abi.m2_attn_decode_kv4(cache, s["q"], H * D, s["out"], H * D, H, s["lens"], D ** -0.5, s["ws"], s["ws"].numel(),
                           stream)
    return s["out"]


# ------------------------------------------------------------------ the plain forms

def _rope_plain(s):
    H, K, D, rot = s["heads"], s["kv_heads"], s["head_dim"], s["rot"]
    x = s["qkv"][:, :(H + K) * D].float().view(-1, H + K, D)
    if s["norm"]:
        w = torch.cat([s["q_w"].float().expand(H, D), s["k_w"].float().expand(K, D)])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if rot:
        i = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
        angle = s["pos"].double()[:, None] * s["theta"] ** (-2.0 * i / rot)
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        r = x[..., :rot]
        if s["pairs"] == "half":
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        x = torch.cat([r, x[..., rot:]], -1)
    x = x.to(torch.bfloat16)
    return x[:, :H].reshape(-1, H * D), x[:, H:].reshape(-1, K * D)


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


def _quantized(x, D):
    """Rows as the cache holds them."""
    g = x.float().view(x.shape[0], -1, D // 16, 16)
    _, scale = _scale_bytes(g.abs().amax(-1, keepdim=True))
    return (_value(_codes(g, scale)) * scale).view(x.shape[0], -1)


def _cache_plain(s):
    K, D = s["kv_heads"], s["head_dim"]
    k, v = _unpack(s["pages"], K, D)
    dev = k.device
    cu_all, cu_new = (torch.tensor(s[c], device=dev) for c in ("cu_all", "cu_new"))
    total, past = s["cu_all"][-1], s["past"].long()
    seq = torch.repeat_interleave(torch.arange(s["nseq"], device=dev), cu_all[1:] - cu_all[:-1], output_size=total)
    at = torch.arange(total, device=dev) - cu_all[seq]
    page = s["table"].long()[seq, at // PAGE]
    fresh = at >= past[seq]
    source = (cu_new[seq] + at - past[seq]).clamp(min=0)

    def rows(old, new):
        old = old[page, :, at % PAGE].reshape(total, K * D)
        return torch.where(fresh[:, None], _quantized(new, D)[source], old).to(torch.bfloat16)
    return rows(k, s["kv"][:, :K * D]), rows(v, s["kv"][:, K * D:])


def _attend(q, k, v, seen):
    """q [n][K][rows][D], k and v [n][K][m][D], seen [n][rows][m]: rows that see nothing are 0."""
    p = torch.matmul(q, k.transpose(-1, -2))
    p.masked_fill_(~seen[:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))


def _prompt_plain(s):
    H, K, D, n = s["heads"], s["kv_heads"], s["head_dim"], s["nseq"]
    dev = s["q"].device
    cu_q, cu_k = torch.tensor(s["cu_q"], device=dev), torch.tensor(s["cu_k"], device=dev)
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    mq, mk = (max(b - a for a, b in zip(s[c], s[c][1:])) for c in ("cu_q", "cu_k"))
    i, j = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    # padded to the longest: [n][K][...]
    q = s["q"][(cu_q[:-1, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))].view(n, mq, K, H // K, D)
    q = (q.permute(0, 2, 1, 3, 4).float() * D ** -0.5).reshape(n, K, mq * (H // K), D)
    at = (cu_k[:-1, None] + j).clamp(max=max(0, s["k"].shape[0] - 1))
    k = s["k"][at].view(n, mk, K, D).transpose(1, 2).float()
    v = s["v"][at].view(n, mk, K, D).transpose(1, 2).float()
    seen = (j <= i[:, None] + (nk - nq)[:, None, None]) & (j < nk[:, None, None])
    out = _attend(q, k, v, seen.repeat_interleave(H // K, 1))
    out = out.view(n, K, mq, H // K, D).permute(0, 2, 1, 3, 4).reshape(n, mq, H * D).to(torch.bfloat16)
    return out[i < nq[:, None]]


def _step_plain(s):
    H, K, D, n = s["heads"], s["kv_heads"], s["head_dim"], s["nseq"]
    k, v = _unpack(s["pages"], K, D)
    at = s["table"].long().clamp(min=0)
    width = at.shape[1] * PAGE
    k = k[at].transpose(1, 2).reshape(n, K, width, D)
    v = v[at].transpose(1, 2).reshape(n, K, width, D)
    q = s["q"].float().view(n, K, H // K, D) * D ** -0.5
    seen = torch.arange(width, device=k.device) < s["lens"][:, None, None]
    return _attend(q, k, v, seen).reshape(n, H * D).to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    plain = {"rope": _rope_plain, "cache": _cache_plain, "prompt": _prompt_plain, "step": _step_plain}
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


def _exact_quantized(x, D):
    """fp64 rows -> the nearest values of the cache, by trying every level."""
    g = x.reshape(-1, 16)
    grid = torch.tensor(sorted({(8 + b % 8) * 2.0 ** (b // 8 - 18) if b > 7 else b * 2.0 ** -17 for b in range(256)}),
                        dtype=torch.float64, device=x.device)
    grid = grid[grid <= 10240.0]
    t = (g.abs().amax(-1) / 6).clamp(max=10240.0)
    hi = torch.searchsorted(grid, t).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    to_lo, to_hi = t - grid[lo], grid[hi] - t
    # grid position parity is the last mantissa bit's
    s = torch.where((to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0)), grid[lo], grid[hi])[:, None]
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    best, least = torch.zeros_like(g), (g.abs()).clone()
    for c in (2, 4, 6, 1, 3, 5, 7):  # the even codes first: ties stay with them
        off = (g.abs() - level[c] * s).abs()
        better = off < least
        best, least = torch.where(better, level[c] * s, best), torch.where(better, off, least)
    return (best * g.sign()).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    H, K, D = s["heads"], s["kv_heads"], s["head_dim"]
    f = torch.float64
    if s["op"] == "rope":
        rot, x = s["rot"], s["qkv"].to(f)
        q, k = x[:, :H * D].reshape(-1, H, D), x[:, H * D:(H + K) * D].reshape(-1, K, D)
        found = []
        for y, w in ((q, s["q_w"]), (k, s["k_w"])):
            if w is not None:
                y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.to(f)
            if rot:
                freq = torch.exp(torch.arange(rot // 2, device=x.device, dtype=f) * (-2 * math.log(s["theta"]) / rot))
                turn = torch.polar(torch.ones_like(freq), s["pos"].to(f)[:, None] * freq)[:, None]
                first = list(range(rot // 2)) if s["pairs"] == "half" else list(range(0, rot, 2))
                second = [i + (rot // 2 if s["pairs"] == "half" else 1) for i in first]
                z = torch.complex(y[..., first], y[..., second]) * turn
                y = y.clone()
                y[..., first], y[..., second] = z.real, z.imag
            found.append(y.reshape(len(y), -1))
        return tuple(found)
    if s["op"] == "cache":
        past = s["past"].tolist()
        ks, vs = [], []
        for i in range(s["nseq"]):
            new = s["kv"][s["cu_new"][i]:s["cu_new"][i + 1]].to(f)
            k, v = _exact_rows(s, i, past[i])
            ks += [k.transpose(0, 1).reshape(past[i], K * D), _exact_quantized(new[:, :K * D], D)]
            vs += [v.transpose(0, 1).reshape(past[i], K * D), _exact_quantized(new[:, K * D:], D)]
        return torch.cat(ks), torch.cat(vs)
    out = torch.zeros(s["q"].shape, dtype=f, device="cuda")
    for i in range(s["nseq"]):
        if s["op"] == "step":
            a, b, n = i, i + 1, int(s["lens"][i])
            k, v = _exact_rows(s, i, n)
        else:
            a, b = s["cu_q"][i], s["cu_q"][i + 1]
            rows = slice(s["cu_k"][i], s["cu_k"][i + 1])
            k = s["k"][rows].to(f).view(-1, K, D).transpose(0, 1)
            v = s["v"][rows].to(f).reshape(-1, K, D).transpose(0, 1)
            n = k.shape[1]
        for h in range(H):
            for r in range(a, b, 2048):  # a block of query rows
                e = min(b, r + 2048)
                score = s["q"][r:e, h * D:(h + 1) * D].to(f) @ k[h // (H // K)].T / math.sqrt(D)
                last = n - b + torch.arange(r, e, device="cuda")  # the last key that a row sees
                score[torch.arange(n, device="cuda") > last[:, None]] = -math.inf
                out[r:e, h * D:(h + 1) * D] = torch.softmax(score, -1) @ v[h // (H // K)]
    return out
