"""Cases of the operators around a decoder layer's attention: a shared prefix, an encoder's states, the residual stream.

Three operators, each in its plain form (elementary torch operations in 32 bits or more) and, where
``own`` is true, through the package's public calls on the same inputs:

  shared    attention of one new token per request over a paged cache in which several requests share a long prefix,
            and have slots of their own behind it (``PagedCache.decode_shared``);
  cross     attention of a decoder's tokens to an encoder's states, of another length and with some of them
            masked (``svx.cross_attn``);
  residual  what lies between two blocks: the norm after a block, its gate, the scaled residual sum and the norm
            before the next one (``svx.residual_norm``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}  # (fp32: the residual stream alone)
EPS = 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four branches of one short prompt on a small Draft: launch latency
        dict(name="shared four branches", op="shared", groups="4", loose=0, prefix="2048", hq=4, hkv=1, d=64, page=16, own_lo=1,
             own_hi=32, dtype="bf16", layout="token"),
        # sixteen samples of one long prompt
        dict(name="shared sixteen samples", op="shared", groups="16", loose=0, prefix="32768", hq=32, hkv=8, d=128, page=64,
             own_lo=1, own_hi=512, dtype="bf16", layout="token"),
        # several prompts, one of them used by one request and one by none, requests without a prefix, some that have
        # nothing of their own yet, pages of 24
        dict(name="shared ragged groups", op="shared", groups="5 1 0 7", loose=2, prefix="777 5000 1200 2999", hq=28,
             hkv=4, d=128, page=24, own_lo=0, own_hi=300, dtype="fp16", layout="head"),
        # a large batch behind one long system prompt: the products bound the prefix, the bytes the rest
        dict(name="shared large batch", op="shared", groups="256", loose=0, prefix="65536", hq=32, hkv=8, d=128, page=128,
             own_lo=1, own_hi=512, dtype="bf16", layout="token"),
        # one token against one encoded input, each query head with keys of its own
        dict(name="cross one token", op="cross", batch=1, n=1, hq=16, hkv=16, d=64, states=1500, len_lo=1500, masked=0.0,
             dtype="fp16", layout="fused"),
        # a decoding batch over states of unequal length, some of them masked, one request without any
        dict(name="cross tokens of a batch", op="cross", batch=32, n=1, hq=32, hkv=8, d=128, states=6404, len_lo=0, masked=0.2,
             dtype="bf16", layout="fused"),
        # prompts against encoded inputs
        dict(name="cross prompts", op="cross", batch=4, n=448, hq=16, hkv=16, d=64, states=1500, len_lo=701, masked=0.0,
             dtype="bf16", layout="heads"),
        # many queries against a few states: the rows of queries and outputs are the bytes
        dict(name="cross short states", op="cross", batch=8, n=4096, hq=16, hkv=16, d=64, states=77, len_lo=20, masked=0.0,
             dtype="fp16", layout="fused"),
        # long against long: the products
        dict(name="cross long", op="cross", batch=1, n=8192, hq=32, hkv=8, d=128, states=16384, len_lo=16384, masked=0.0,
             dtype="bf16", layout="fused"),
        # one token between two blocks, with a gated block
        dict(name="residual one token", op="residual", rows=1, d=4096, post=False, gate="scalar", act="tanh", stream="bf16",
             alpha=1.0, beta=1.0, dtype="bf16"),
        # an odd batch, a residual stream in 32 bits, norms on both sides, a gate per channel
        dict(name="residual odd batch", op="residual", rows=777, d=5128, post=True, gate="channel", act="none", stream="fp32",
             alpha=1.0, beta=0.22, dtype="fp16"),
        # a long prompt, norms on both sides, a gate per element
        dict(name="residual long prompt", op="residual", rows=32768, d=4096, post=True, gate="element", act="sigmoid",
             stream="bf16", alpha=0.9, beta=1.1, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(numbers):
    return " ".join(map(str, numbers))


def _numbers(text):
    return [int(x) for x in text.split()]


def draw(rng):
    op = rng.choice(["shared", "shared", "cross", "cross", "residual"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "residual":
        d = 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, max(1, min(32768, (1 << 27) // d))), d=d, post=rng.random() < 0.5,
                    gate=rng.choice(["none", "scalar", "channel", "element"]), act=rng.choice(["none", "tanh", "sigmoid"]),
                    stream=rng.choice([dtype, dtype, "fp32"]), alpha=rng.choice([1.0, rng.uniform(0.5, 1.5)]),
                    beta=rng.choice([1.0, rng.uniform(0.1, 1.5)]), dtype=dtype)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 7, 8, 12])
    if op == "shared":
        n = rng.choice([1, 1, 2, 3, 5])
        groups = [_log(rng, 1, max(1, 192 // n)) for _ in range(n)]
        if n > 2:
            groups[rng.randrange(n)] = 0
        batch = sum(groups)
        # products of the prefixes, and elements of K, as far as the listed cases go
        most = max(1, min(65536, 32768 * 8 * 128 // (n * hkv * d), (1 << 33) // (batch * hkv * group * d)))
        prefix = [_log(rng, 1, most) for _ in range(n)]
        own = _log(rng, 1, max(1, min(4096, 32768 * 8 * 128 // (batch * hkv * d))))
        return dict(op=op, groups=_text(groups), loose=rng.choice([0, 0, 1, 3]), prefix=_text(prefix), hq=hkv * group, hkv=hkv, d=d,
                    page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128]), own_lo=rng.choice([0, 1, own // 2, own]), own_hi=own,
                    dtype=dtype, layout=rng.choice(["token", "head"]))
    batch = _log(rng, 1, 64)
    states = _log(rng, 1, max(1, min(32768, 32768 * 8 * 128 // (batch * hkv * d))))
    few = rng.random() < 0.4
    most = max(1, min(8192, (1 << 38) // (batch * hkv * group * d * states), (1 << 27) // (batch * hkv * group * d)))
    return dict(op=op, batch=batch, n=_log(rng, 1, 8) if few else _log(rng, 1, most), hq=hkv * group, hkv=hkv, d=d, states=states,
                len_lo=rng.choice([0, states // 2, states, states]), masked=rng.choice([0.0, 0.0, 0.3]), dtype=dtype,
                layout=rng.choice(["fused", "heads"]))


def _spread(lo, hi, n):
    """n lengths evenly from lo to hi, the long and the short mixed."""
    even = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    return even[::2] + even[1::2][::-1]


def _own_lengths(c):
    return _spread(c["own_lo"], c["own_hi"], sum(_numbers(c["groups"])) + c["loose"])


def _state_lengths(c):
    return _spread(c["len_lo"], c["states"], c["batch"])


def work(c):
    size = 2  # of an element
    if c["op"] == "shared":
        used = [(n, p) for n, p in zip(_numbers(c["groups"]), _numbers(c["prefix"])) if n]
        slots = sum(p for _, p in used) + sum(_own_lengths(c))
        batch = sum(_numbers(c["groups"])) + c["loose"]
        rows = sum(n * p for n, p in used) + sum(_own_lengths(c))
        return {"bytes": slots * c["hkv"] * 2 * size * c["d"] + batch * c["hq"] * (2 * size * c["d"] + 4),
                "flops": 4 * rows * c["hq"] * c["d"]}
    if c["op"] == "cross":
        states = sum(_state_lengths(c))
        rows = c["batch"] * c["n"] * c["hq"]
        return {"bytes": states * c["hkv"] * 2 * size * c["d"] + (c["batch"] * c["states"] if c["masked"] else 0) +
                rows * (2 * size * c["d"] + 4), "flops": 4 * c["n"] * states * c["hq"] * c["d"]}
    stream = 4 if c["stream"] == "fp32" else 2
    n = c["rows"] * c["d"]
    return {"bytes": n * (2 * size + 2 * stream + (size if c["gate"] == "element" else 0)), "flops": 12 * n}


# ------------------------------------------------------------------ inputs

def _pool(g, pages, c, dtype, dev):
    """K or V pages: [page][slot][KV head][d], held in that order or (layout "head") with the heads outside the slots."""
    if c["layout"] == "head":
        return torch.randn((pages, c["hkv"], c["page"], c["d"]), generator=g, device=dev, dtype=dtype).transpose(1, 2)
    return torch.randn((pages, c["page"], c["hkv"], c["d"]), generator=g, device=dev, dtype=dtype)


def _spoil(s, table, lens, page):
    """Slots behind a length hold whatever was there before: the worst is not a number."""
    room = table.shape[1] * page
    lens = torch.tensor(lens, device=table.device)
    row, slot = (torch.arange(room, device=table.device)[None, :] >= lens[:, None]).nonzero(as_tuple=True)
    at = table[row, slot // page].long()
    mine = at >= 0
    for pool in ("k", "v"):
        s[pool][at[mine], (slot % page)[mine]] = float("nan")


def _tables(g, lens, page, dev):
    """Page tables of several sets of sequences over one pool: pages in random order, as an allocator leaves them; -1
    behind each sequence's own."""
    need = [[-(-n // page) for n in part] for part in lens]
    total = sum(map(sum, need)) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    tables, at = [], 0
    for part in need:
        wide = max(part + [1])
        count = torch.tensor(part, device=dev)[:, None]
        col = torch.arange(wide, device=dev)[None, :]
        first = at + torch.cumsum(count, 0) - count
        tables.append(torch.where(col < count, order[(first + col).clamp(max=total - 1)], -1).to(torch.int32).contiguous())
        at += sum(part)
    return tables, total


def _inputs(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    s = {"case": dict(c)}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if c["op"] == "shared":
        groups, prefix, own_lens = _numbers(c["groups"]), _numbers(c["prefix"]), _own_lengths(c)
        batch = len(own_lens)
        s["first"] = ints([sum(groups[:i]) for i in range(len(groups) + 1)])
        s["prefix_lens"], s["lens"] = ints(prefix), ints(own_lens)
        (s["prefix_table"], s["table"]), pages = _tables(g, [prefix, own_lens], c["page"], dev)
        s["k"], s["v"] = _pool(g, pages, c, dt, dev), _pool(g, pages, c, dt, dev)
        _spoil(s, s["prefix_table"], prefix, c["page"])
        _spoil(s, s["table"], own_lens, c["page"])
        s["q"] = 2 * torch.randn((batch, c["hq"], 1, c["d"]), generator=g, device=dev, dtype=dt)
        s["o"] = torch.zeros((batch, c["hq"], 1, c["d"]), device=dev, dtype=dt)
        s["lse"] = torch.zeros((batch, c["hq"], 1), device=dev)
        return s
    if c["op"] == "cross":
        b, n, hq, hkv, d, t = c["batch"], c["n"], c["hq"], c["hkv"], c["d"], c["states"]
        lens = _state_lengths(c)
        s["lens"] = ints(lens) if c["len_lo"] < t else None
        hidden = torch.arange(t, device=dev)[None, :] >= torch.tensor(lens, device=dev)[:, None]
        s["mask"] = None
        if c["masked"]:
            s["mask"] = torch.rand((b, t), generator=g, device=dev) >= c["masked"]
            hidden = hidden | ~s["mask"]
        if c["layout"] == "fused":  # the projections' outputs: k and v side by side, q and o with a token's heads together
            kv = torch.randn((b, t, 2, hkv, d), generator=g, device=dev, dtype=dt)
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
            s["q"] = (2 * torch.randn((b, n, hq, d), generator=g, device=dev, dtype=dt)).transpose(1, 2)
            s["o"] = torch.zeros((b, n, hq, d), device=dev, dtype=dt).transpose(1, 2)
        else:  # states laid out once by head
            s["k"], s["v"] = (torch.randn((b, hkv, t, d), generator=g, device=dev, dtype=dt).transpose(1, 2) for _ in range(2))
            s["q"] = 2 * torch.randn((b, hq, n, d), generator=g, device=dev, dtype=dt)
            s["o"] = torch.zeros((b, hq, n, d), device=dev, dtype=dt)
        s["k"][hidden], s["v"][hidden] = float("nan"), float("nan")
        s["lse"] = torch.zeros((b, hq, n), device=dev)
        return s
    rows, d, st = c["rows"], c["d"], DTYPES[c["stream"]]
    s["h"] = 4 * torch.randn((rows, d), generator=g, device=dev, dtype=st)
    s["y"] = torch.randn((rows, d), generator=g, device=dev, dtype=dt)
    s["norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
    s["post_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt) if c["post"] else None
    shape = {"none": None, "scalar": (1,), "channel": (d,), "element": (rows, d)}[c["gate"]]
    s["gate"] = None if shape is None else torch.randn(shape, generator=g, device=dev, dtype=dt)
    s["h_out"] = torch.zeros((rows, d), device=dev, dtype=st)
    s["x"] = torch.zeros((rows, d), device=dev, dtype=dt)
    return s


def prepare(c, seed):
    s = _inputs(c, seed)
    if own:  # the handles that a program keeps beside these tensors
        from speculative_decoding_verification_chunked_gb300 import svx
        s["svx"] = svx
        if c["op"] == "shared":
            s["cache"] = svx.PagedCache(s["k"], s["v"])
    return s


# ------------------------------------------------------------------ the plain forms

def _slots(pool, table, lens, page):
    """[sequence][KV head][slot][d] in 32 bits, zero behind a sequence's length."""
    table = table.long().clamp(min=0)
    n, room = table.shape[0], table.shape[1] * page
    live = torch.arange(room, device=table.device)[None, :] < lens[:, None]
    rows = pool[table].reshape(n, room, pool.shape[2], pool.shape[3])
    return torch.where(live[:, :, None, None], rows, 0.0).transpose(1, 2).float(), live


def _shared(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    group, scale = hq // hkv, 1.0 / math.sqrt(c["d"])
    batch = s["q"].shape[0]
    q = s["q"].float().reshape(batch, hkv, group, d) * scale
    k, live = _slots(s["k"], s["table"], s["lens"], page)
    score = torch.matmul(q, k.transpose(2, 3)).masked_fill(~live[:, None, None, :], float("-inf"))
    v, _ = _slots(s["v"], s["table"], s["lens"], page)
    o = torch.zeros((batch, hkv, group, d), device=q.device)
    lse = torch.zeros((batch, hkv, group), device=q.device)
    begin, groups = 0, _numbers(c["groups"])
    for i, n in enumerate(groups + [c["loose"]]):
        if not n:
            continue
        at = slice(begin, begin + n)
        begin += n
        mine = [score[at]]
        if i < len(groups):
            # [KV head][request, query head][d] against the prefix, once for all of them
            pk, there = _slots(s["k"], s["prefix_table"][i:i + 1], s["prefix_lens"][i:i + 1], page)
            rows = q[at].transpose(0, 1).reshape(hkv, n * group, d)
            far = torch.matmul(rows, pk[0].transpose(1, 2)).masked_fill(~there[0], float("-inf"))
            mine.append(far.reshape(hkv, n, group, -1).transpose(0, 1))
            del pk, far
        top = torch.stack([x.amax(-1) for x in mine]).amax(0)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))[..., None]
        p = torch.exp(mine[0] - top)
        total, sums = p.sum(-1), torch.matmul(p, v[at])
        if len(mine) > 1:
            p = torch.exp(mine[1] - top)
            del mine
            pv, _ = _slots(s["v"], s["prefix_table"][i:i + 1], s["prefix_lens"][i:i + 1], page)
            total = total + p.sum(-1)
            sums = sums + torch.matmul(p.transpose(0, 1).reshape(hkv, n * group, -1), pv[0]).reshape(hkv, n, group, d).transpose(0, 1)
        o[at] = sums / torch.where(total > 0, total, torch.ones_like(total))[..., None]
        lse[at] = top[..., 0] + total.log()
    return {"o": o.reshape(batch, hq, 1, d).to(s["o"].dtype), "lse": lse.reshape(batch, hq, 1)}


def _cross(s):
    c = s["case"]
    b, n, hq, hkv, d = c["batch"], c["n"], c["hq"], c["hkv"], c["d"]
    group = hq // hkv
    live = torch.ones((b, c["states"]), dtype=torch.bool, device=s["q"].device)
    if s["lens"] is not None:
        live = torch.arange(c["states"], device=live.device)[None, :] < s["lens"][:, None]
    if s["mask"] is not None:
        live = live & s["mask"]
    o, lse = torch.zeros_like(s["o"]), torch.zeros_like(s["lse"])
    step = max(1, min(hkv, (1 << 28) // (b * group * n * c["states"])))  # KV heads at a time: their scores take room
    for h in range(0, hkv, step):
        m = min(step, hkv - h)
        heads = slice(h * group, (h + m) * group)
        k = torch.where(live[:, :, None, None], s["k"][:, :, h:h + m], 0.0).transpose(1, 2).float()
        q = s["q"][:, heads].float().reshape(b, m, group * n, d)
        score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
        score = score.masked_fill(~live[:, None, None, :], float("-inf"))
        top = score.amax(-1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        p = torch.exp(score - top)
        del score
        total = p.sum(-1, keepdim=True)
        v = torch.where(live[:, :, None, None], s["v"][:, :, h:h + m], 0.0).transpose(1, 2).float()
        rows = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
        o[:, heads] = rows.reshape(b, m * group, n, d).to(o.dtype)
        lse[:, heads] = (top + total.log()).reshape(b, m * group, n)
    return {"o": o, "lse": lse}


def _residual(s):
    c = s["case"]
    y = s["y"].float()
    if c["post"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post_norm"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        if c["act"] == "tanh":
            gate = (torch.exp(2 * gate) - 1) / (torch.exp(2 * gate) + 1)
        elif c["act"] == "sigmoid":
            gate = 1 / (1 + torch.exp(-gate))
        y = y * gate
    h = c["alpha"] * s["h"].float() + c["beta"] * y
    x = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["norm"].float()
    return {"h": h.to(s["h"].dtype), "x": x.to(s["y"].dtype)}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if not own:
        return {"shared": _shared, "cross": _cross, "residual": _residual}[c["op"]](s)
    if c["op"] == "shared":
        s["cache"].decode_shared(s["q"], s["prefix_table"], s["prefix_lens"], s["first"], s["table"], s["lens"], s["o"], s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "cross":
        s["svx"].cross_attn(s["q"], s["k"], s["v"], s["o"], s["lse"], lens=s["lens"], mask=s["mask"])
        return {"o": s["o"], "lse": s["lse"]}
    s["svx"].residual_norm(s["h"], s["y"], s["h_out"], s["x"], norm=s["norm"], eps=EPS, post_norm=s["post_norm"],
                           post_eps=EPS if c["post"] else None, gate=s["gate"], act=None if c["act"] == "none" else c["act"],
                           alpha=c["alpha"], beta=c["beta"])
    return {"h": s["h_out"], "x": s["x"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _sequence(pool, row, n, page, head):
    """The first n slots of a sequence, one KV head: [n][d] in 64 bits."""
    return pool[row[:-(-n // page)].long()][:, :, head].reshape(-1, pool.shape[3])[:n].double()


def _exact_shared(c, s):
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    group, prefix, own_lens = hq // hkv, _numbers(c["prefix"]), _own_lengths(c)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["o"].device)
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device=o.device)
    bounds = s["first"].tolist()
    for h in range(hkv):
        heads = slice(h * group, (h + 1) * group)
        for i in range(len(bounds)):
            begin = bounds[i]
            end = bounds[i + 1] if i + 1 < len(bounds) else len(own_lens)  # the last ones have no prefix
            if end == begin:
                continue
            z_far = None
            if i < len(prefix):
                pk, pv = (_sequence(s[x], s["prefix_table"][i], prefix[i], page, h) for x in "kv")
                z_far = torch.einsum("bgd,td->bgt", s["q"][begin:end, heads, 0].double(), pk) / d ** 0.5
                ln_far = torch.logsumexp(z_far, -1)
                o_far = torch.softmax(z_far, -1) @ pv
            for b in range(begin, end):
                parts, outs = [], []
                if z_far is not None:
                    parts.append(ln_far[b - begin])
                    outs.append(o_far[b - begin])
                if own_lens[b]:
                    ok, ov = (_sequence(s[x], s["table"][b], own_lens[b], page, h) for x in "kv")
                    z = s["q"][b, heads, 0].double() @ ok.T / d ** 0.5
                    parts.append(torch.logsumexp(z, -1))
                    outs.append(torch.softmax(z, -1) @ ov)
                if parts:
                    both = torch.logsumexp(torch.stack(parts), 0)
                    lse[b, heads, 0] = both
                    o[b, heads, 0] = sum(torch.exp(p - both)[:, None] * x for p, x in zip(parts, outs))
    return {"o": o, "lse": lse}


def _exact_cross(c, s):
    group, d = c["hq"] // c["hkv"], c["d"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["o"].device)
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device=o.device)
    for b, n in enumerate(_state_lengths(c)):
        seen = torch.arange(n, device=o.device)
        if s["mask"] is not None:
            seen = s["mask"][b, :n].nonzero()[:, 0]
        if not len(seen):
            continue
        for h in range(c["hq"]):
            k, v = (s[x][b, seen, h // group].double() for x in "kv")
            z = s["q"][b, h].double() @ k.T / d ** 0.5
            lse[b, h] = torch.logsumexp(z, -1)
            o[b, h] = torch.softmax(z, -1) @ v
    return {"o": o, "lse": lse}


def _exact_residual(c, s):
    y = s["y"].double()
    if c["post"]:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["d"] + EPS) * s["post_norm"].double()
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    if s["gate"] is not None and c["act"] != "none":
        gate = torch.tanh(gate) if c["act"] == "tanh" else torch.sigmoid(gate)
    h = s["h"].double() * c["alpha"] + y * gate * c["beta"]
    return {"h": h, "x": h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / c["d"] + EPS) * s["norm"].double()}


def exact(c, seed):
    s = _inputs(c, seed)
    return {"shared": _exact_shared, "cross": _exact_cross, "residual": _exact_residual}[c["op"]](c, s)
