"""Values that show a single lost or doubled token: every channel of a kv head is zero but for a few tokens, so that
each of these is a part of the output far above the tolerances of rounding, however long the sequence."""
import torch


def cover(v, cu, Hkv, D, step, every):
    """v [T][Hkv * D] in place.  Tokens next to a multiple of `step` (both sides, and the first and the last one) get a
    channel in every head; or, `every`, each token gets one channel of one head.  Returns the largest number of tokens
    that share a channel."""
    most = 0
    for a, b in zip(cu, cu[1:]):
        n = b - a
        if n == 0:
            continue
        x = v[a:b].zero_().view(n, Hkv, D)
        if every:
            i = torch.arange(n, device=v.device)
            slot = i % (Hkv * D)
            x[i, slot // D, slot % D] = 1.0 + 0.5 * (i % 3).to(v.dtype)  # (levels of the 4-bit format)
            most = max(most, -(-n // (Hkv * D)))
        else:
            edge = torch.arange(0, n + step, step)
            i = torch.cat([edge - 1, edge])
            i = torch.cat([i[(i >= 0) & (i < n)], torch.tensor([0, n - 1])]).unique().to(v.device)
            c = torch.arange(len(i), device=v.device)
            for h in range(Hkv):
                x[i, h, (c * 5 + h) % D] = 1.0 + 0.5 * (c % 3).to(v.dtype)
            most = max(most, -(-len(i) // D))
    return most
