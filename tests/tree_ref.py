"""Plain 64-bit forms of the operators for trees of drafted tokens, for the tests: the
rules of include/mamba2.h, one node at a time."""
import torch

F = torch.float64


def paths(parent):
    """The path of every node (its own index last); an empty one for a node that is not part of the tree."""
    out = []
    for r, p in enumerate(parent):
        if p == -1:
            out.append([r])
        elif 0 <= p < r and out[p]:
            out.append(out[p] + [r])
        else:
            out.append([])
    return out


def conv(ring, pos, x, w, bias, parent, silu):
    """ring [L][C], x [n][C] -> (out, size) [n][C], size = sum of |terms| before the activation."""
    L = ring.shape[0]
    out, size = torch.zeros(x.shape, dtype=F, device=x.device), torch.zeros(x.shape, dtype=F, device=x.device)
    w = w.to(F)
    for r, path in enumerate(paths(parent)):
        if not path:
            continue
        line = [x[k].to(F) for k in path[-(L + 1):]]
        line = [ring[(pos - 1 - k) % L].to(F) for k in range(L + 1 - len(line))][::-1] + line
        b = torch.zeros_like(line[0]) if bias is None else bias.to(F)
        v = b + sum(t * w[:, j] for j, t in enumerate(line))
        size[r] = b.abs() + sum((t * w[:, j]).abs() for j, t in enumerate(line))
        out[r] = v * torch.sigmoid(v) if silu else v
    return out, size


def steps(dt_raw, dt_bias, A_log):
    dt = torch.nn.functional.softplus(dt_raw.to(F) + dt_bias.to(F), threshold=1e9).clamp(1e-9, 1e9)
    return dt, torch.exp(-dt * torch.exp(A_log.to(F)))


def ssm_step(h, x, B, dt, dA):
    """h [H][P][N], x [H][P], B [G][N], dt and dA [H]."""
    B = B.to(F).repeat_interleave(h.shape[0] // B.shape[0], 0)
    return dA[:, None, None] * h + (dt[:, None] * x.to(F))[..., None] * B[:, None]


def ssm(h, x, B, C, dt_raw, dt_bias, A_log, D, parent):
    """h [H][P][N] fp32, x [n][H][P], B and C [n][G][N] -> (y, size) [n][H][P]; size: the sum of |terms|."""
    H = h.shape[0]
    dt, dA = steps(dt_raw, dt_bias, A_log)
    y, size = torch.zeros(x.shape, dtype=F, device=x.device), torch.zeros(x.shape, dtype=F, device=x.device)
    states = {}
    for r, path in enumerate(paths(parent)):
        if not path:
            continue
        s, a = states[path[-2]] if len(path) > 1 else (h.to(F), h.to(F).abs())
        s, a = ssm_step(s, x[r], B[r], dt[r], dA[r]), ssm_step(a, x[r].abs(), B[r].abs(), dt[r], dA[r])
        states[r] = s, a
        c = C[r].to(F).repeat_interleave(H // C.shape[1], 0)[:, None]
        y[r] = (s * c).sum(-1) + D.to(F)[:, None] * x[r].to(F)
        size[r] = (a * c.abs()).sum(-1) + (D.to(F)[:, None] * x[r].to(F)).abs()
    return y, size


def verify(p, q, parent, token, u, u_next):
    """The walk with every remainder normalised: (path, token)."""
    V = p.shape[1]

    def clean(row):
        row = row.to(F)
        return torch.where((row > 0) & row.isfinite(), row, torch.zeros_like(row))
    if not parent or parent[0] != -1:
        return [], -1
    path, rest = [0], clean(p[0])
    for r in range(1, len(parent)):
        x = token[r]
        if parent[r] != path[-1] or not 0 <= x < V:
            continue
        d = None if q is None else clean(q[path[-1]])
        if u[r] * (1.0 if d is None else float(d[x])) < float(rest[x]):
            path.append(r)
            rest = clean(p[r])
            continue
        if d is None:
            rest = rest.clone()
            rest[x] = 0.0
        else:
            rest = (rest - d).clamp(min=0)
        if float(rest.sum()) > 0:
            rest = rest / rest.sum()
    if float(rest.sum()) <= 0:
        rest = clean(p[path[-1]])
    if float(rest.sum()) <= 0:
        return path, -1
    total = rest.cumsum(0)
    at = int((total <= u_next * total[-1]).sum())
    return path, min(at, V - 1)


def attend(q, k, v, scale, context, parent):
    """q [n][H][D]; k, v [context + n][Hkv][D] -> (out, weight, sum, score); a node sees the context and its path.
    weight = sum p |v|, sum = sum |v| over what it sees, score = the largest sum of |terms| of a score."""
    n, H, D = q.shape
    G = H // k.shape[1]
    out = torch.zeros(q.shape, dtype=F, device=q.device)
    size, total, score = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out[..., :1])
    for r, path in enumerate(paths(parent)):
        see = list(range(context)) + [context + a for a in path if context + a < k.shape[0]]
        if not path or not see:
            continue
        kk, vv = k[see].to(F).repeat_interleave(G, 1), v[see].to(F).repeat_interleave(G, 1)
        s = torch.einsum("hd,thd->ht", q[r].to(F) * scale, kk)
        w = torch.softmax(s, -1)
        out[r], size[r] = torch.einsum("ht,thd->hd", w, vv), torch.einsum("ht,thd->hd", w, vv.abs())
        total[r] = vv.abs().sum(0)
        score[r] = torch.einsum("hd,thd->ht", q[r].to(F).abs() * abs(scale), kk.abs()).amax(-1, keepdim=True)
    return out, size, total, score


def random_parents(n, rng, kind="tree"):
    """Parents of n nodes: "chain", "star" (all below node 0), "tree", "forest" (several nodes follow the context)."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    low = -1 if kind == "forest" else 0
    return [-1] + [rng.randint(max(low, r - 6), r - 1) if r > 1 else low + 0 * r for r in range(1, n)]


def ancestors_sum(parent, la):
    """Sums of la [n][H] along the paths (for tolerances)."""
    out = torch.zeros_like(la)
    for r, path in enumerate(paths(parent)):
        if path:
            out[r] = la[path].sum(0)
    return out


