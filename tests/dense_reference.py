"""The dense cache operators from their definitions, in 64 bits (torch, any device).

Written from the formulas alone: which tokens a query sees, where it and they sit, one
softmax, one weighted mean; eviction as a stable sort.  Shares nothing with the library.
"""

import torch

D = 128


def rotate(x, pos, base):
    """Rows x [..., 128] turned to positions pos (broadcast over the leading axes)."""
    i = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    a = torch.as_tensor(pos, dtype=torch.float64, device=x.device)[..., None] * base ** (-2.0 * i / D)
    u, v = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()], dim=-1)


def tokens(pool, table, page):
    """A paged pool [pages][H][page][128] as [B][H][tokens][128]."""
    return torch.stack([torch.cat([pool[int(pg)] for pg in row], dim=1) for row in table.cpu()])


def positions(L, n, causal, own):
    return [L - n + i + int(own) for i in range(n)] if causal else [L] * n


def weights_of(q, k, p, base, scale, sinks=0, window=0, token_positions=False):
    """Softmax weights [rows][L] of query rows q [rows][128], all at position p, over keys k [L][128]."""
    L = k.shape[0]
    t = torch.arange(L, device=k.device)
    kr = rotate(k, t, base)
    s = scale * rotate(q, p, base) @ kr.T
    seen = t < p
    if window:
        far = t < p - window
        sink = t < sinks
        at = p if token_positions else min(p, sinks + window)
        s = torch.where(far & sink, scale * rotate(q, at, base) @ kr.T, s)
        seen = seen & (~far | sink)
    if not bool(seen.any()):
        return torch.zeros_like(s)
    return torch.softmax(torch.where(seen, s, torch.full_like(s, -torch.inf)), dim=-1)


def attend(q, k, v, lens, G, base=1.0e6, scale=None, causal=False, own=False, want_weights=False, **view):
    """q [B][n][Hq][128], k and v [B][H][cap][128] -> out [B][n][Hq][128] fp64 (or the weights
    each slot receives, [B][H][cap])."""
    B, n, Hq, _ = q.shape
    H = Hq // G
    scale = scale or D ** -0.5
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=q.device)
    got = torch.zeros(B, H, k.shape[2], dtype=torch.float64, device=q.device)
    for b in range(B):
        L = int(lens[b])
        for i, p in enumerate(positions(L, n, causal, own)):
            if p <= 0:
                continue
            for h in range(H):
                w = weights_of(q[b, i, h * G:(h + 1) * G].double(), k[b, h, :L].double(), p, base, scale, **view)
                got[b, h, :L] += w.sum(0)
                seen = (w > 0).any(0)
                out[b, i, h * G:(h + 1) * G] = w[:, seen] @ v[b, h, :L][seen].double()
    return got if want_weights else out


def evict(w, L, keep, sinks, recent):
    """Kept slots (ascending list) of one head's weights w [>= L]."""
    if L <= keep:
        return list(range(L))
    free = list(range(sinks, L - recent))
    x = [float(v) for v in w[sinks:L - recent].double().tolist()]
    order = sorted(range(len(free)), key=lambda j: (x[j] != x[j], -x[j] if x[j] == x[j] else 0.0, j))
    best = [free[j] for j in order[:keep - sinks - recent]]
    return sorted(list(range(sinks)) + best + list(range(L - recent, L)))
