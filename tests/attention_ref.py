"""Plain 64-bit forms of the attention operators, for the tests: the formulas of
include/mamba2.h, one step at a time, in torch doubles."""
import math

import torch

F = torch.float64
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the scale bytes that a finite group can get, by byte: 4 significant bits, e = 0 subnormal, at most 10240
SCALES = [b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(256)]
TOP_BYTE = SCALES.index(10240.0)


def nearest_even(x, grid):
    """Index of the nearest grid value (ascending); ties to the even index."""
    hi = torch.searchsorted(grid, x).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = x - grid[lo], grid[hi] - x
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantize(x):
    """Rows [..., D] -> (codes uint8, scale bytes uint8 [..., D/16]); a NaN makes its group's byte 255."""
    g = x.to(F).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    bad = g.isnan().any(-1)
    m = torch.where(g.isnan(), torch.zeros_like(g), g).abs().amax(-1)
    grid = torch.tensor(SCALES[:TOP_BYTE + 1], dtype=F, device=x.device)
    byte = nearest_even((m / 6).clamp(max=10240.0), grid)
    s = grid[byte]
    lev = torch.tensor(LEVELS, dtype=F, device=x.device)
    ratio = torch.where(s[..., None] > 0, g.abs() / s[..., None], torch.zeros_like(g)).clamp(max=6.0)
    code = nearest_even(torch.where(ratio.isnan(), torch.zeros_like(ratio), ratio), lev)
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    code = code + 8 * (g < 0)
    return code.to(torch.uint8).view(x.shape), torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)


def dequantize(code, byte):
    lev = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=F, device=code.device)
    sc = torch.tensor(SCALES[:248] + [math.nan] * 8, dtype=F, device=code.device)
    return lev[code.long()] * sc[byte.long()].repeat_interleave(16, -1)


def rounded_rows(x):
    return dequantize(*quantize(x))


def pack_block(kc, kb, vc, vb):
    """Codes [64][D] and scale bytes [64][D/16] of one page and head -> its 72 * D bytes, byte by byte."""
    D = kc.shape[1]
    out = torch.zeros(72 * D, dtype=torch.uint8)
    kc, kb, vc, vb = (t.cpu().to(torch.int64) for t in (kc, kb, vc, vb))
    for t in range(64):
        for d in range(D):
            g, c, h, n = d // 16, d % 16 // 4, d % 4 // 2, d % 2
            out[t * (D // 2) + c * (D // 8) + g * 2 + h] |= int(kc[t, d]) << (4 * n)
            i, r = d // 8, d % 8
            out[32 * D + t // 8 * 4 * D + r * (D // 2) + t % 8 // 2 * (D // 8) + i] |= int(vc[t, d]) << (4 * (t % 2))
        for g in range(D // 16):
            out[64 * D + t * (D // 16) + g] = int(kb[t, g])
            out[68 * D + t // 2 * (D // 8) + g // 2 * 4 + t % 2 * 2 + g % 2] = int(vb[t, g])
    return out


def rope(x, w, pos, theta, rot, interleaved, eps):
    """x [T][heads][D] -> (y, size): y in 64 bits, and |a| + |b| of every pair (what rounding errors scale with)."""
    y = x.to(F)
    if w is not None:
        y = y * w.to(F) / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    size = y.abs()
    if rot:
        i = torch.arange(rot // 2, dtype=F, device=x.device)
        ang = pos.to(F)[:, None] * theta ** (-2.0 * i / rot)
        cos, sin = ang.cos()[:, None], ang.sin()[:, None]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y, size = y.clone(), size.clone()
        y[..., a], y[..., b] = ya * cos - yb * sin, yb * cos + ya * sin
        size[..., a] = size[..., b] = ya.abs() + yb.abs()
    return y, size


def attend(q, k, v, scale, first_seen=None):
    """q [nq][H][D], k and v [nk][Hkv][D], query j sees keys 0 .. j + nk - nq (all of them if first_seen is
    "all").  Returns (out, weight), weight = sum p |v|; rows that see nothing are 0."""
    nq, H, D = q.shape
    nk, G = k.shape[0], H // k.shape[1]
    out = torch.zeros(nq, H, D, dtype=F, device=q.device)
    size = torch.zeros_like(out)
    if nq == 0 or nk == 0:
        return out, size
    last = torch.arange(nq, device=q.device) + nk - nq
    if first_seen == "all":
        last = torch.full_like(last, nk - 1)
    seen = torch.arange(nk, device=q.device) <= last[:, None]
    for h in range(H):
        s = (q[:, h].to(F) * scale) @ k[:, h // G].to(F).T
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        m = s.amax(-1, keepdim=True)
        p = torch.where(seen, torch.exp(s - torch.where(last[:, None] >= 0, m, torch.zeros_like(m))),
                        torch.zeros_like(s))
        p = p / torch.where(last[:, None] >= 0, p.sum(-1, keepdim=True), torch.ones_like(m))
        vh = v[:, h // G].to(F)
        if vh.isfinite().all():
            out[:, h], size[:, h] = p @ vh, p @ vh.abs()
        else:  # a value that a row does not see must not reach it
            t = torch.where(seen[..., None], p[..., None] * vh, torch.zeros((), dtype=F, device=q.device))
            out[:, h], size[:, h] = t.sum(1), t.abs().sum(1)
    return out, size
