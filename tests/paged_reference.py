"""Plain 64-bit implementations of the paged-cache operators for the tests, from their definitions: loops over
requests and heads in float64, sharing nothing with the CUDA path."""
import numpy as np
import torch


def rotate64(x, pos, inv_freq, neighbours, scale=1.0):
    """x: float64 [n][heads][d], pos: ints [n]."""
    half = len(inv_freq)
    ang = torch.as_tensor(pos, dtype=torch.float64)[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(ang)[:, None] * scale, torch.sin(ang)[:, None] * scale
    out = x.clone()
    ia = torch.arange(half) * 2 if neighbours else torch.arange(half)
    ib = ia + (1 if neighbours else half)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def heads64(x, w, eps, pos, inv_freq, neighbours, scale=1.0):
    """Normed and rotated heads, and |y_a| + |y_b| of each element's pair (the size its fp32 error goes by)."""
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
    return rotate64(y, pos, inv_freq, neighbours, scale), pair_size(y, len(inv_freq), neighbours)


def pair_size(y, half, neighbours):
    size = y.abs()
    ia = torch.arange(half) * 2 if neighbours else torch.arange(half)
    ib = ia + (1 if neighbours else half)
    both = size[..., ia] + size[..., ib]
    size = size.clone()
    size[..., ia], size[..., ib] = both, both
    return size


def rows_of(pages, table_row, n):
    """The first n slots of a request, [n][Hkv][d]."""
    size = pages.shape[1]
    return torch.stack([pages[int(table_row[t // size]), t % size] for t in range(n)]) if n else pages[:0, 0]


def decode64(q, k_pages, v_pages, table, lens, scale, acc=None):
    """o, lse, acc + weights, and per row what the error bounds go by: sum w|v| and max_t scale sum|q k|."""
    B, Hq, _, d = q.shape
    hkv = k_pages.shape[2]
    G = Hq // hkv
    o, lse = torch.zeros(B, Hq, 1, d, dtype=torch.float64), torch.full((B, Hq, 1), -np.inf, dtype=torch.float64)
    size, spread = torch.zeros(B, Hq, 1, d, dtype=torch.float64), torch.zeros(B, Hq, 1, dtype=torch.float64)
    out = None if acc is None else acc.double().clone()
    w_all = None if acc is None else torch.zeros_like(out)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k, v = rows_of(k_pages, table[b], n).double(), rows_of(v_pages, table[b], n).double()
        for h in range(Hq):
            x, kk, vv = q[b, h, 0].double(), k[:, h // G], v[:, h // G]
            s = (kk @ x) * scale
            m = s.max()
            if m == -np.inf:
                continue
            p = torch.exp(s - m)
            w = p / p.sum()
            o[b, h, 0], lse[b, h, 0] = w @ vv, m + torch.log(p.sum())
            size[b, h, 0], spread[b, h, 0] = w @ vv.abs(), (kk.abs() @ x.abs()).max() * scale
            if out is not None:
                out[b, h // G, :n] += w
                w_all[b, h // G, :n] += w
    return o, lse, out, size, spread, w_all


def evict64(acc, pos, length, next_pos, budget, sink, recent):
    """One row: the new order of its first min(length, budget) slots, as old slots."""
    n = min(length, budget)
    def preference(t):
        protected = pos[t] < sink or pos[t] >= next_pos - recent
        weight = -np.inf if np.isnan(acc[t]) else float(acc[t])
        return (0 if protected else 1, -weight if not protected else 0.0, t)
    kept = set(sorted(range(length), key=preference)[:n])
    spares = iter(sorted(t for t in kept if t >= n))
    return [t if t in kept else next(spares) for t in range(n)]
