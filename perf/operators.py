"""Cases of the paged-cache operators: what a Draft's one-token step and the entry of a verification round cost.

Three operators, each in its plain form (elementary torch operations in 32 bits or more) and, where
``own`` is true, through the package's public calls on the same inputs:

  heads    norms of query and key heads with the position rotation, into a round's dense tensors or into a
           paged cache (``svx.qk_norm_rope``, ``PagedCache.append``);
  decode   attention of one new token per request over a paged cache, with or without the accumulated
           attention weight of every cached token (``PagedCache.decode``);
  evict    keeping the slots of a paged cache with the largest accumulated weights (``PagedCache.evict``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
THETA = 1.0e6
EPS = 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a Draft's step for one request: the latency of a single token's heads
        dict(name="heads one token", op="heads", dest="pages", batch=1, n=1, hq=32, hkv=8, d=128, rot=128,
             pairs="halves", norm=True, dtype="bf16", page=16, start=1000, ragged=False),
        # a round's queries and candidates: a 16-node token tree for each of 8 requests
        dict(name="heads token tree", op="heads", dest="dense", batch=8, n=16, hq=32, hkv=8, d=128, rot=128,
             pairs="halves", norm=True, dtype="bf16", page=0, start=65536, ragged=False),
        # prompts of unequal length into the cache, rotated in part and in neighbouring pairs, no norms
        dict(name="heads ragged prompts", op="heads", dest="pages", batch=5, n=777, hq=12, hkv=3, d=64, rot=32,
             pairs="neighbours", norm=False, dtype="fp16", page=24, start=131, ragged=True),
        # a whole long prompt
        dict(name="heads long prompt", op="heads", dest="pages", batch=1, n=32768, hq=32, hkv=8, d=128, rot=128,
             pairs="halves", norm=True, dtype="bf16", page=64, start=0, ragged=False),
        # one token over a short cache: launch latency
        dict(name="decode short", op="decode", batch=1, hq=4, hkv=1, d=64, dtype="bf16", page=16, len_lo=512,
             len_hi=512, weights=False, layout="token"),
        # a ragged batch, one request still empty, seven query heads to a KV head, pages of 24
        dict(name="decode ragged", op="decode", batch=5, hq=28, hkv=4, d=128, dtype="fp16", page=24, len_lo=0,
             len_hi=2999, weights=False, layout="head"),
        # a Draft batch that accumulates the weights it evicts by
        dict(name="decode with weights", op="decode", batch=16, hq=32, hkv=8, d=128, dtype="bf16", page=64,
             len_lo=1, len_hi=8192, weights=True, layout="token"),
        # one long request, weights accumulated
        dict(name="decode one long", op="decode", batch=1, hq=32, hkv=8, d=128, dtype="bf16", page=16,
             len_lo=131072, len_hi=131072, weights=True, layout="token"),
        # eight requests of equal length, the largest batch
        dict(name="decode eight long", op="decode", batch=8, hq=32, hkv=8, d=128, dtype="bf16", page=128,
             len_lo=32768, len_hi=32768, weights=False, layout="token"),
        # the Draft's cache went over its budget by one page: the step that is taken over and over
        dict(name="evict a page", op="evict", batch=8, hkv=8, d=128, dtype="bf16", page=64, length=2112,
             budget=2048, sink=4, recent=256),
        # a small cache with one KV head
        dict(name="evict small", op="evict", batch=2, hkv=1, d=64, dtype="fp16", page=24, length=777, budget=512,
             sink=0, recent=100),
        # after a long prompt: the cache goes down to its budget at once
        dict(name="evict after prompt", op="evict", batch=8, hkv=8, d=128, dtype="bf16", page=16, length=32768,
             budget=4096, sink=4, recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["heads", "decode", "decode", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    batch = _log(rng, 1, 64)
    most = 32768 * 8 * 128  # elements of K of a drawn cache (the largest listed one has eight times as many)
    if op == "heads":
        group = min(group, 8)
        n = _log(rng, 1, max(1, min(16384, most // (batch * hkv * d * group))))
        rot = rng.choice([d, d, d // 2])
        return dict(op=op, dest=rng.choice(["pages", "dense"]), batch=batch, n=n, hq=hkv * group, hkv=hkv, d=d, rot=rot,
                    pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7, dtype=dtype, page=page,
                    start=_log(rng, 1, 20000) - 1 if n == 1 and batch <= 4 else rng.randrange(2000),
                    ragged=rng.random() < 0.3)
    length = _log(rng, 1 if op == "decode" else 64, max(64, min(131072, most // (batch * hkv * d))))
    if op == "decode":
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, dtype=dtype, page=page,
                    len_lo=rng.choice([0, 1, length // 2, length]), len_hi=length, weights=rng.random() < 0.5,
                    layout=rng.choice(["token", "head"]))
    budget = max(1, int(length * rng.uniform(0.1, 1.1)))
    sink = rng.choice([0, 1, 4])
    sink = min(sink, budget - 1)
    return dict(op=op, batch=batch, hkv=hkv, d=d, dtype=dtype, page=page, length=length, budget=budget, sink=sink,
                recent=int((budget - sink) * rng.uniform(0.0, 0.5)))


def _lengths(c):
    """The cached lengths of a case's requests: evenly spread from len_lo to len_hi, the long and the short mixed."""
    lo, hi, n = c["len_lo"], c["len_hi"], c["batch"]
    even = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    return even[::2] + even[1::2][::-1]


def _new_tokens(c):
    """How many of its n tokens each request of a heads case brings."""
    n, b = c["n"], c["batch"]
    return [n - (n * i) // b for i in range(b)] if c["ragged"] else [n] * b


def work(c):
    if c["op"] == "heads":
        t = sum(_new_tokens(c))
        heads = c["hq"] + 2 * c["hkv"]
        meta = t * (4 + (8 * c["hkv"] if c["dest"] == "pages" else 0))
        return {"bytes": 2 * 2 * t * heads * c["d"] + meta, "flops": 10 * t * (c["hq"] + c["hkv"]) * c["d"]}
    if c["op"] == "decode":
        t = sum(_lengths(c)) * c["hkv"]
        return {"bytes": t * (4 * c["d"] + (8 if c["weights"] else 0)) + 4 * c["batch"] * c["hq"] * (c["d"] + 1),
                "flops": 4 * t * (c["hq"] // c["hkv"]) * c["d"]}
    rows, n, keep = c["batch"] * c["hkv"], c["length"], min(c["budget"], c["length"])
    moved = keep * (n - keep) // n  # kept slots behind the budget, if the kept ones lie evenly
    return {"bytes": rows * (8 * n + 8 * keep + moved * 2 * 2 * 2 * c["d"]), "flops": 2 * rows * n}


# ------------------------------------------------------------------ inputs

def _pool(g, pages, c, dtype, dev):
    """K or V pages: [page][slot][KV head][d], held in that order or (layout "head") with the heads outside the slots."""
    if c.get("layout") == "head":
        return torch.randn((pages, c["hkv"], c["page"], c["d"]), generator=g, device=dev, dtype=dtype).transpose(1, 2)
    return torch.randn((pages, c["page"], c["hkv"], c["d"]), generator=g, device=dev, dtype=dtype)


def _table(g, lens, page, dev):
    """Pages in random order, as an allocator leaves them; -1 behind each request's own."""
    need = [-(-n // page) for n in lens]
    wide, total = max(max(need), 1), sum(need) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    col = torch.arange(wide, device=dev)[None, :]
    need_t = torch.tensor(need, device=dev)[:, None]
    first = torch.cumsum(need_t, 0) - need_t
    table = torch.where(col < need_t, order[(first + col).clamp(max=total - 1)], -1).to(torch.int32)
    return table.contiguous(), total


def _inputs(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    s = {"case": dict(c)}
    if c["op"] == "heads":
        b, n, hq, hkv, d = c["batch"], c["n"], c["hq"], c["hkv"], c["d"]
        # the projection's output: q, k and v heads side by side
        s["qkv"] = torch.randn((b, n, hq + 2 * hkv, d), generator=g, device=dev, dtype=dt) * 2
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
            s["k_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
        start = [max(0, c["start"] - 17 * i) for i in range(b)]
        s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        gone = torch.randint(0, 30000, (b, 1), generator=g, device=dev)  # tokens that the cache no longer holds
        step = torch.arange(n, device=dev)[None, :]
        if c["dest"] == "dense":
            step = (step + 1).float().log2().long()  # a tree node's depth
        s["pos"] = (s["start"][:, None] + gone + step).to(torch.int32).contiguous()
        s["new"] = torch.tensor(_new_tokens(c), dtype=torch.int32, device=dev) if c["ragged"] else None
        s["q_out"] = torch.zeros((b, hq, n, d), device=dev, dtype=dt)
        if c["dest"] == "dense":
            s["k_out"] = torch.zeros((b, n, hkv, d), device=dev, dtype=dt)
            s["v_out"] = torch.zeros((b, n, hkv, d), device=dev, dtype=dt)
        else:
            s["table"], pages = _table(g, [x + n for x in start], c["page"], dev)
            s["k"], s["v"] = _pool(g, pages, c, dt, dev), _pool(g, pages, c, dt, dev)
            room = s["table"].shape[1] * c["page"]
            s["acc"] = torch.rand((b, hkv, room), generator=g, device=dev)
            s["slot_pos"] = torch.arange(room, device=dev, dtype=torch.int32).expand(b, hkv, room).contiguous()
        return s
    if c["op"] == "decode":
        b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
        lens = _lengths(c)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["table"], pages = _table(g, lens, c["page"], dev)
        s["k"], s["v"] = _pool(g, pages, c, dt, dev), _pool(g, pages, c, dt, dev)
        room = s["table"].shape[1] * c["page"]
        # slots behind a request's last token hold whatever was there before: the worst is not a number
        row, slot = (torch.arange(room, device=dev)[None, :] >= s["lens"][:, None]).nonzero(as_tuple=True)
        at = s["table"][row, slot // c["page"]].long()
        mine = at >= 0
        s["k"][at[mine], (slot % c["page"])[mine]] = float("nan")
        s["v"][at[mine], (slot % c["page"])[mine]] = float("nan")
        s["q"] = 2 * torch.randn((b, hq, 1, d), generator=g, device=dev, dtype=dt)
        s["o"] = torch.zeros((b, hq, 1, d), device=dev, dtype=dt)
        s["lse"] = torch.zeros((b, hq, 1), device=dev)
        if c["weights"]:
            s["acc"] = torch.rand((b, hkv, room), generator=g, device=dev) ** 4
            s["acc_out"] = torch.zeros((b, hkv, room), device=dev)
        return s
    b, hkv, n = c["batch"], c["hkv"], c["length"]
    lens = [max(1, n - 5 * i) for i in range(b)]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["table"], pages = _table(g, lens, c["page"], dev)
    s["k"], s["v"] = _pool(g, pages, c, dt, dev), _pool(g, pages, c, dt, dev)
    room = s["table"].shape[1] * c["page"]
    # weights: most tokens hardly attended to, some never (equal weights), a few strongly
    w = torch.rand((b, hkv, room), generator=g, device=dev)
    s["acc"] = torch.where(w < 0.1, torch.zeros_like(w), w ** 8 * 20).contiguous()
    # positions: increasing with gaps (earlier evictions), the newest ones in arbitrary slots
    gap = torch.randint(1, 3, (b, hkv, room), generator=g, device=dev)
    pos = torch.cumsum(gap, -1) - 1
    # (slots that earlier evictions filled from behind: neighbours of a random order change places)
    key = torch.arange(room, device=dev) + 64 * torch.rand((b, hkv, room), generator=g, device=dev)
    s["slot_pos"] = torch.gather(pos, -1, torch.argsort(key, -1)).to(torch.int32).contiguous()
    s["next_pos"] = (s["slot_pos"].amax((1, 2)) + 1).to(torch.int32)
    s["acc_out"] = torch.zeros((b, hkv, room), device=dev)
    s["pos_out"] = torch.zeros((b, hkv, room), device=dev, dtype=torch.int32)
    s["len_out"] = torch.zeros(b, device=dev, dtype=torch.int32)
    return s


def _inv_freq(rot):
    return [THETA ** (-2.0 * i / rot) for i in range(rot // 2)]


def prepare(c, seed):
    s = _inputs(c, seed)
    if own:  # the handles that a program keeps beside these tensors
        from speculative_decoding_verification_chunked_gb300 import svx
        s["svx"] = svx
        if c["op"] == "heads":
            s["rope"] = svx.Rope(c["rot"], inv_freq=_inv_freq(c["rot"]), neighbours=c["pairs"] == "neighbours")
        if "k" in s:
            s["cache"] = svx.PagedCache(s["k"], s["v"])
    return s


# ------------------------------------------------------------------ the plain forms

def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, pos, rot, pairs):
    """x: [b, n, heads, d] in 32 bits; pos: [b, n].  Angles in 64 bits: positions reach far."""
    inv = torch.tensor(_inv_freq(rot), dtype=torch.float64, device=x.device)
    angle = pos.double()[..., None] * inv
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs == "halves":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, rest), -1)


def _heads(s):
    c = s["case"]
    b, n, hq, hkv = c["batch"], c["n"], c["hq"], c["hkv"]
    dt = DTYPES[c["dtype"]]
    qkv = s["qkv"]
    q = _rotate(_norm(qkv[:, :, :hq], s["q_norm"]), s["pos"], c["rot"], c["pairs"]).to(dt).transpose(1, 2)
    k = _rotate(_norm(qkv[:, :, hq:hq + hkv], s["k_norm"]), s["pos"], c["rot"], c["pairs"]).to(dt)
    v = qkv[:, :, hq + hkv:]
    here = torch.ones((b, n), dtype=torch.bool, device=q.device)
    if s["new"] is not None:
        here = torch.arange(n, device=q.device)[None, :] < s["new"][:, None]
    q_out = torch.where(here[:, None, :, None], q, s["q_out"])
    if c["dest"] == "dense":
        rows = here[:, :, None, None]
        return {"q": q_out, "k": torch.where(rows, k, s["k_out"]), "v": torch.where(rows, v, s["v_out"])}
    row, tok = here.nonzero(as_tuple=True)
    slot = s["start"][row].long() + tok
    page, at = s["table"][row, slot // c["page"]].long(), slot % c["page"]
    s["k"][page, at] = k[row, tok]
    s["v"][page, at] = v[row, tok]
    s["acc"][row, :, slot] = 0.0
    s["slot_pos"][row, :, slot] = s["pos"][row, tok][:, None].expand(-1, hkv)
    return {"q": q_out, "k": s["k"], "v": s["v"], "acc": s["acc"], "slot_pos": s["slot_pos"]}


def _decode(s):
    c = s["case"]
    b, hq, hkv, d, page = c["batch"], c["hq"], c["hkv"], c["d"], c["page"]
    lens, table = s["lens"], s["table"].long().clamp(min=0)
    room = table.shape[1] * page
    live = torch.arange(room, device=lens.device)[None, :] < lens[:, None]
    # [b, hkv, slot, d], zero behind the last token
    rows = live[:, None, :, None]
    k = torch.where(rows, s["k"][table].reshape(b, room, hkv, d).transpose(1, 2), 0.0).float()
    q = s["q"].float().reshape(b, hkv, hq // hkv, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    score = score.masked_fill(~live[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(rows, s["v"][table].reshape(b, room, hkv, d).transpose(1, 2), 0.0).float()
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    out = {"o": o.reshape(b, hq, 1, d).to(DTYPES[c["dtype"]]), "lse": (top + total.log()).reshape(b, hq, 1)}
    if c["weights"]:
        w = (p / torch.where(total > 0, total, torch.ones_like(total))).sum(2)
        out["acc"] = torch.where(live[:, None, :], s["acc"] + w, s["acc_out"])
    return out


def _evict(s):
    c = s["case"]
    b, hkv, page, budget = c["batch"], c["hkv"], c["page"], c["budget"]
    lens, acc, pos = s["lens"], s["acc"], s["slot_pos"]
    room = acc.shape[-1]
    slot = torch.arange(room, device=acc.device).expand(b, hkv, room)
    live = slot < lens[:, None, None]
    kept_len = lens.clamp(max=budget)
    always = (pos < c["sink"]) | (pos >= (s["next_pos"] - c["recent"])[:, None, None])
    weight = torch.where(torch.isnan(acc), float("-inf"), acc)
    # slots in order of preference: always kept, then by weight, then by slot; those behind the length last
    order = torch.sort(weight, dim=-1, descending=True, stable=True).indices
    rank = torch.gather(torch.where(live, torch.where(always, 0, 1), 2), -1, order)
    order = torch.gather(order, -1, torch.sort(rank, dim=-1, stable=True).indices)
    kept = torch.zeros_like(live).scatter(-1, order, slot < kept_len[:, None, None])
    # the kept slots behind the new length, in order, fill the evicted ones before it, in order
    before = slot < kept_len[:, None, None]
    hole, spare = before & ~kept, ~before & kept
    spares = torch.sort((~spare).to(torch.int8), dim=-1, stable=True).indices
    source = torch.where(hole, torch.gather(spares, -1, (torch.cumsum(hole, -1) - 1).clamp(min=0)), slot)
    acc_out = torch.where(before, torch.gather(acc, -1, source), s["acc_out"])
    pos_out = torch.where(before, torch.gather(pos, -1, source), s["pos_out"])
    row, head, to = hole.nonzero(as_tuple=True)
    fro = source[row, head, to]
    p_to, p_fro = s["table"][row, to // page].long(), s["table"][row, fro // page].long()
    for pool in (s["k"], s["v"]):
        pool[p_to, to % page, head] = pool[p_fro, fro % page, head]
    return {"acc": acc_out, "pos": pos_out, "len": kept_len.to(torch.int32), "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if not own:
        return {"heads": _heads, "decode": _decode, "evict": _evict}[c["op"]](s)
    if c["op"] == "heads":
        qkv, hq, hkv = s["qkv"], c["hq"], c["hkv"]
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        eps = EPS if c["norm"] else None
        if c["dest"] == "dense":
            s["svx"].qk_norm_rope(q, k, v, s["pos"], s["rope"], s["q_out"], s["k_out"], s["v_out"], q_norm=s["q_norm"],
                                  k_norm=s["k_norm"], eps=eps, n_new=s["new"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        s["cache"].append(q, k, v, s["pos"], s["rope"], s["table"], s["start"], s["q_out"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=eps, n_new=s["new"], acc=s["acc"], slot_pos=s["slot_pos"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "acc": s["acc"], "slot_pos": s["slot_pos"]}
    if c["op"] == "decode":
        if c["weights"]:
            s["cache"].decode(s["q"], s["table"], s["lens"], s["o"], s["lse"], acc_in=s["acc"], acc_out=s["acc_out"])
            return {"o": s["o"], "lse": s["lse"], "acc": s["acc_out"]}
        s["cache"].decode(s["q"], s["table"], s["lens"], s["o"], s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    s["cache"].evict(s["table"], s["lens"], c["budget"], c["sink"], c["recent"], s["next_pos"], s["acc"], s["slot_pos"],
                     s["acc_out"], s["pos_out"], s["len_out"])
    return {"acc": s["acc_out"], "pos": s["pos_out"], "len": s["len_out"], "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_heads(c, s):
    hq, hkv, rot, d = c["hq"], c["hkv"], c["rot"], c["d"]
    x = s["qkv"].double()
    turn = torch.exp(-math.log(THETA) * torch.arange(0, rot, 2, dtype=torch.float64, device=x.device) / rot)
    phase = torch.polar(torch.ones_like(turn), torch.zeros_like(turn))[None, None] * 1j
    phase = torch.exp(phase * (s["pos"].double()[:, :, None] * turn))[:, :, None]  # e^{i pos f}

    def heads(part, w):
        if w is not None:
            part = part / torch.sqrt(part.pow(2).sum(-1, keepdim=True) / d + EPS) * w.double()
        if c["pairs"] == "halves":
            z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:rot].contiguous()) * phase
            turned = torch.cat((z.real, z.imag), -1)
        else:
            z = torch.view_as_complex(part[..., :rot].reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * phase
            turned = torch.view_as_real(z).reshape(*part.shape[:-1], rot)
        return torch.cat((turned, part[..., rot:]), -1)

    q, k, v = heads(x[:, :, :hq], s["q_norm"]), heads(x[:, :, hq:hq + hkv], s["k_norm"]), x[:, :, hq + hkv:]
    new = _new_tokens(c)
    q_out = s["q_out"].double()
    if c["dest"] == "dense":
        k_out, v_out = s["k_out"].double(), s["v_out"].double()
        for b, n in enumerate(new):
            q_out[b, :, :n] = q[b, :n].transpose(0, 1)
            k_out[b, :n], v_out[b, :n] = k[b, :n], v[b, :n]
        return {"q": q_out, "k": k_out, "v": v_out}
    pool_k, pool_v, acc, slot_pos = s["k"].double(), s["v"].double(), s["acc"].double(), s["slot_pos"].clone()
    page = c["page"]
    for b, n in enumerate(new):
        q_out[b, :, :n] = q[b, :n].transpose(0, 1)
        first = int(s["start"][b])
        flat = (s["table"][b].long()[:, None] * page + torch.arange(page, device=x.device)).reshape(-1)[first:first + n]
        pool_k.view(-1, hkv, d)[flat] = k[b, :n]
        pool_v.view(-1, hkv, d)[flat] = v[b, :n]
        acc[b, :, first:first + n] = 0
        slot_pos[b, :, first:first + n] = s["pos"][b, :n]
    return {"q": q_out, "k": pool_k, "v": pool_v, "acc": acc, "slot_pos": slot_pos}


def _exact_decode(c, s):
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    group = hq // hkv
    o, lse = torch.zeros_like(s["o"], dtype=torch.float64), torch.full_like(s["lse"], float("-inf"), dtype=torch.float64)
    acc = s["acc_out"].double() if c["weights"] else None
    for b, n in enumerate(_lengths(c)):
        if not n:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            k, v = (s[x][pages][:, :, h].reshape(-1, d)[:n].double() for x in "kv")
            z = s["q"][b, h * group:(h + 1) * group, 0].double() @ k.T / d ** 0.5
            ln = torch.logsumexp(z, -1)
            w = torch.exp(z - ln[:, None])
            o[b, h * group:(h + 1) * group, 0] = w @ v
            lse[b, h * group:(h + 1) * group, 0] = ln
            if acc is not None:
                acc[b, h, :n] = s["acc"][b, h, :n].double() + w.sum(0)
    out = {"o": o, "lse": lse}
    if acc is not None:
        out["acc"] = acc
    return out


def _exact_evict(c, s):
    import numpy as np
    page, budget = c["page"], c["budget"]
    acc, pos = s["acc"].cpu().numpy().astype(np.float64), s["slot_pos"].cpu().numpy()
    acc_out, pos_out = s["acc_out"].cpu().numpy().astype(np.float64), s["pos_out"].cpu().numpy()
    lens, nxt, table = s["lens"].tolist(), s["next_pos"].tolist(), s["table"].cpu().numpy()
    moves = []
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(c["hkv"]):
            a, q = acc[b, h, :n], pos[b, h, :n]
            must = (q < c["sink"]) | (q >= nxt[b] - c["recent"])
            # last key first: must, then weight, then the lower slot
            best = np.lexsort((np.arange(n), -np.where(np.isnan(a), -np.inf, a), ~must))[:m]
            keep = set(best.tolist())
            here = np.arange(m)
            here[[t for t in range(m) if t not in keep]] = sorted(t for t in keep if t >= m)
            acc_out[b, h, :m], pos_out[b, h, :m] = a[here], q[here]
            moves += [(table[b, t // page], t % page, table[b, f // page], f % page, h) for t, f in enumerate(here.tolist()) if f != t]
    k, v = s["k"].clone(), s["v"].clone()
    if moves:
        p1, t1, p0, t0, h = torch.tensor(np.array(moves, dtype=np.int64), device=k.device).T
        k[p1, t1, h], v[p1, t1, h] = s["k"][p0, t0, h], s["v"][p0, t0, h]
    return {"acc": acc_out, "pos": pos_out, "len": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32), "k": k, "v": v}


def exact(c, seed):
    s = _inputs(c, seed)
    return {"heads": _exact_heads, "decode": _exact_decode, "evict": _exact_evict}[c["op"]](c, s)
