"""Plain 64-bit implementations of the attention operators for the tests, from their definitions, sharing nothing with the CUDA
path: one softmax over the keys that count."""
import math

import torch


def attend64(q, k, v, scale):
    """One group of rows: q [rows][d], k, v [keys][d].  o, lse, and what the error bounds go by: sum w|v| and max scale sum|q k|."""
    q, k, v = q.double(), k.double(), v.double()
    rows, d = q.shape
    if k.shape[0] == 0:
        zero = torch.zeros((rows, d), dtype=torch.float64, device=q.device)
        return zero, torch.full((rows,), -math.inf, dtype=torch.float64, device=q.device), zero, zero[:, 0]
    s = (q @ k.T) * scale
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    w = p / total
    return w @ v, (m + torch.log(total))[:, 0], w @ v.abs(), (q.abs() @ k.abs().T).amax(-1) * scale


def near(o, lse, want, p_error, keys, min_normal=None):
    """o, lse of a group against attend64's.  p_error: relative error of a softmax weight in the product with V.  Bounds: a score is off
    by at most 2^-19 S (S = scale max sum |q k|), an exponential by 2^-21, sums of n terms by n 2^-24."""
    wo, wl, size, spread = want
    u = torch.finfo(o.dtype).eps / 2
    e = spread * 2.0 ** -19
    c = 2 * (e + p_error + keys * 2.0 ** -24)
    bound = wo.abs() * u + size * c[:, None] * (1 + u) + torch.finfo(o.dtype).tiny * torch.finfo(o.dtype).eps
    off = (o.double() - wo).abs()
    assert (off <= bound).all(), f"o: {float((off / bound).max()):.3f} times the bound"
    none = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse), none) and (o[none] == 0).all()
    off = (lse.double() - wl).abs()[~none]
    bound = (e + 2.0 ** -20 + keys * 2.0 ** -24 + wl.abs() * 2.0 ** -22)[~none]
    assert (off <= bound).all(), f"lse: {float((off / bound).max()):.3f} times the bound"


def slots_of(pool, row, n):
    """The first n slots of a page table's row: [n][KV heads][d]."""
    page = pool.shape[1]
    t = torch.arange(n, device=pool.device)
    return pool[row.to(pool.device).long()[t // page], t % page]
