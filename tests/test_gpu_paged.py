"""The paged-cache operators on the GPU against plain 64-bit implementations.

Error bounds, derived before any run.  u = torch.finfo(type).eps / 2 is a rounding to the output type.
  heads   fp32 throughout, one rounding.  The norm's sum of d squares, its square root and three products stay under
          2^-19 relative; the angle is exact to 2^-22 and sine and cosine to 2^-21, together under 2^-20, so a
          rotated value is off by at most (|y_a| + |y_b|) (2^-19 + 2^-20) before its rounding: |z| u + (|y_a| + |y_b|) 2^-18.
  decode  a score (natural units) is off by at most 2^-19 S, S = scale max sum |q_i k_i| (8 tensor-core steps, each
          within 2^-22 of the running size); p keeps 16 bits in two pieces (2^-16 relative, the exponential
          2^-21); sums of n terms within n 2^-24.  So O is off by |O| u + c sum w|v| with
          c = 2 (2^-19 S + 2^-15 + n 2^-24), LSE by 2^-19 S + 2^-20 + n 2^-24 + |LSE| 2^-22, and a weight by c w plus two
          roundings of acc (2^-23 |acc|).
  evict   moves values and compares them: exact.
"""
import numpy as np
import pytest
import torch

from paged_reference import decode64, evict64, heads64

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def unit(t):
    return torch.finfo(t).eps / 2


def make_pool(g, n_pages, page, hkv, d, dtype, layout="token"):
    if layout == "token":
        return torch.randn((n_pages, page, hkv, d), generator=g, dtype=torch.float32).to(dtype).cuda()
    if layout == "head":
        return torch.randn((n_pages, hkv, page, d), generator=g).to(dtype).cuda().transpose(1, 2)
    both = torch.randn((n_pages, 2, page, hkv, d), generator=g).to(dtype).cuda()  # K and V side by side
    return both[:, 0], both[:, 1]


def make_table(g, lens, page, extra=0):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


# ------------------------------------------------------------------ heads

HEADS = [  # b, n, hq, hkv, d, rot, neighbours, norm, type, scale
    (1, 1, 4, 1, 64, 64, False, True, "bf16", 1.0),
    (1, 1, 32, 8, 128, 128, False, True, "bf16", 1.0),
    (3, 5, 6, 2, 128, 64, True, True, "fp16", 1.0),
    (2, 7, 5, 5, 64, 16, True, False, "bf16", 0.75),
    (2, 33, 8, 1, 128, 128, True, True, "fp16", 1.0),
    (1, 700, 40, 8, 128, 128, False, True, "bf16", 1.0),   # several heads per group of lanes
    (4, 1500, 12, 3, 64, 32, False, True, "fp16", 1.0),
    (2, 9, 4, 2, 128, 0, False, True, "bf16", 1.0),        # norms alone
    (256, 1, 2, 1, 64, 64, False, True, "bf16", 1.0),
]


def heads_inputs(case, seed=0, far=200000):
    b, n, hq, hkv, d, rot, nb, norm, ty, scale = case
    g = torch.Generator().manual_seed(seed)
    t = TYPES[ty]
    qkv = (3 * torch.randn((b, n, hq + 2 * hkv, d), generator=g)).to(t)
    qkv[0, 0, 0] = 0  # a head of zeros: the norm's eps alone
    pos = torch.randint(0, far, (b, n), generator=g, dtype=torch.int32)
    wq = wk = None
    if norm:
        wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(t) for _ in range(2))
    inv = [1e5 ** (-2.0 * i / rot) for i in range(rot // 2)]
    return qkv, pos, wq, wk, inv


def heads_reference(case, qkv, pos, wq, wk, inv):
    b, n, hq, hkv, d, rot, nb, norm, ty, scale = case
    eps = 1e-6 if norm else None
    flat = qkv.reshape(b * n, hq + 2 * hkv, d)
    p = pos.reshape(-1)
    q, qs = heads64(flat[:, :hq], wq, eps, p, inv, nb, scale)
    k, ks = heads64(flat[:, hq:hq + hkv], wk, eps, p, inv, nb, scale)
    shape = lambda x: x.reshape(b, n, -1, d)  # noqa: E731
    return shape(q), shape(qs), shape(k), shape(ks), qkv[:, :, hq + hkv:]


def near(got, want, size, t):
    err = (got.double().cpu() - want).abs()
    bound = want.abs() * unit(t) + size * 2.0 ** -18 + torch.finfo(t).tiny * torch.finfo(t).eps
    assert (err <= bound).all(), f"{float((err / bound.clamp(min=1e-30)).max()):.3f} times the bound"


@pytest.mark.parametrize("case", HEADS, ids=str)
def test_heads_dense(svx, case):
    b, n, hq, hkv, d, rot, nb, norm, ty, scale = case
    qkv, pos, wq, wk, inv = heads_inputs(case)
    t = TYPES[ty]
    x = qkv.cuda()
    qo, ko, vo = (torch.full(s, 7.0, dtype=t, device="cuda") for s in ((b, hq, n, d), (b, n, hkv, d), (b, n, hkv, d)))
    cu = lambda w: None if w is None else w.cuda()  # noqa: E731
    svx.qk_norm_rope(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos.cuda(),
                     svx.Rope(rot, inv_freq=inv, neighbours=nb, scale=scale), qo, ko, vo, q_norm=cu(wq), k_norm=cu(wk),
                     eps=1e-6 if norm else None)
    q, qs, k, ks, v = heads_reference(case, qkv, pos, wq, wk, inv)
    near(qo.transpose(1, 2), q, qs, t)
    near(ko, k, ks, t)
    assert torch.equal(vo.cpu(), v)


@pytest.mark.parametrize("layout", ["token", "head", "pair"])
@pytest.mark.parametrize("case", HEADS[1:5] + HEADS[6:7], ids=str)
def test_append(svx, case, layout):
    """Into pages that end anywhere, tokens of unequal number per request, everything else left as it was."""
    b, n, hq, hkv, d, rot, nb, norm, ty, scale = case
    qkv, pos, wq, wk, inv = heads_inputs(case, seed=1)
    t = TYPES[ty]
    g = torch.Generator().manual_seed(2)
    page = 5
    start = torch.randint(0, 23, (b,), generator=g, dtype=torch.int32)
    new = torch.randint(0, n + 1, (b,), generator=g, dtype=torch.int32)
    new[0] = n
    table, total = make_table(g, [int(s) + n for s in start], page, extra=1)
    if layout == "pair":
        kp, vp = make_pool(g, total, page, hkv, d, t, layout)
    else:
        kp, vp = (make_pool(g, total, page, hkv, d, t, layout) for _ in range(2))
    k0, v0 = kp.cpu().clone(), vp.cpu().clone()
    cache = svx.PagedCache(kp, vp)
    room = table.shape[1] * page
    acc = torch.rand((b, hkv, room), device="cuda")
    sp = torch.randint(0, 99, (b, hkv, room), device="cuda", dtype=torch.int32)
    acc0, sp0 = acc.cpu().clone(), sp.cpu().clone()
    x, qo = qkv.cuda(), torch.full((b, hq, n, d), 7.0, dtype=t, device="cuda")
    cu = lambda w: None if w is None else w.cuda()  # noqa: E731
    cache.append(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos.cuda(),
                 svx.Rope(rot, inv_freq=inv, neighbours=nb, scale=scale), table.cuda(), start.cuda(), qo, q_norm=cu(wq),
                 k_norm=cu(wk), eps=1e-6 if norm else None, n_new=new.cuda(), acc=acc, slot_pos=sp)
    assert not cache.check()
    q, qs, k, ks, v = heads_reference(case, qkv, pos, wq, wk, inv)
    want_k, want_v, size = k0.double(), v0.clone(), torch.zeros(k0.shape, dtype=torch.float64)
    for i in range(b):
        m = int(new[i])
        near(qo[i, :, :m].transpose(0, 1), q[i, :m], qs[i, :m], t)
        assert (qo[i, :, m:] == 7.0).all()
        for j in range(m):
            s = int(start[i]) + j
            pg = int(table[i, s // page])
            want_k[pg, s % page], want_v[pg, s % page], size[pg, s % page] = k[i, j], v[i, j], ks[i, j]
            acc0[i, :, s], sp0[i, :, s] = 0.0, pos[i, j]
    near(kp, want_k, size, t)
    untouched = size.amax(-1) == 0
    assert torch.equal(kp.cpu()[untouched], k0[untouched])
    assert torch.equal(vp.cpu(), want_v) and torch.equal(acc.cpu(), acc0) and torch.equal(sp.cpu(), sp0)


def test_far_and_negative_positions_keep_their_phase(svx):
    """The phase is exact for any 32-bit position: 64-bit angles of the reference lose 2^31 2^-53, nothing next to 2^-25."""
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1, 131071]], dtype=torch.int32)
    x = torch.randn((1, 8, 3, 128), generator=torch.Generator().manual_seed(3)).half()
    inv = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    qo, ko = torch.empty((1, 1, 8, 128), dtype=torch.float16, device="cuda"), torch.empty((1, 8, 1, 128), dtype=torch.float16, device="cuda")
    xc = x.cuda()
    svx.qk_norm_rope(xc[:, :, :1], xc[:, :, 1:2], None, pos.cuda(), svx.Rope(128), qo, ko, eps=None)
    q, qs = heads64(x[0, :, :1], None, None, pos[0], inv, False)
    near(qo[0].transpose(0, 1), q, qs, torch.float16)


# ------------------------------------------------------------------ decode

DECODE = [  # lens, hq, hkv, d, page, type, layout, weights
    ((1,), 1, 1, 64, 1, "bf16", "token", True),
    ((0,), 4, 2, 128, 16, "bf16", "token", True),
    ((512,), 4, 1, 64, 16, "bf16", "token", False),
    ((0, 1, 15, 16, 17, 31, 32, 33), 8, 2, 128, 16, "bf16", "token", True),
    ((127, 128, 129, 0, 1000), 14, 2, 128, 24, "fp16", "head", True),     # 7 heads to a KV head, pages inside tiles
    ((300, 5), 27, 3, 64, 7, "fp16", "pair", True),                       # 9: the wide form
    ((700, 0, 61), 32, 2, 128, 100, "bf16", "head", True),                # 16
    ((260, 33), 40, 1, 64, 32, "bf16", "token", True),                    # 40: three blocks of heads
    ((90, 450), 17, 1, 128, 16, "bf16", "token", True),                   # 17: a block of one
    ((5000,), 8, 1, 128, 64, "fp16", "token", True),                      # one item over many CTAs
    ((2500, 1, 0, 1800), 8, 8, 64, 16, "bf16", "token", False),           # one head each
    (tuple(range(0, 256)), 2, 1, 64, 8, "bf16", "token", True),           # the most requests
]


def decode_inputs(case, seed=0, q_scale=2.0, extra=1):
    lens, hq, hkv, d, page, ty, layout, weights = case
    g = torch.Generator().manual_seed(seed)
    t = TYPES[ty]
    table, total = make_table(g, lens, page, extra=extra)
    if layout == "pair":
        kp, vp = make_pool(g, total, page, hkv, d, t, layout)
    else:
        kp, vp = (make_pool(g, total, page, hkv, d, t, layout) for _ in range(2))
    # what lies behind a length, and pages of nobody, hold the worst
    used = torch.zeros((total, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for s in range(n):
            used[int(table[b, s // page]), s % page] = True
    k64, v64 = kp.cpu().clone(), vp.cpu().clone()
    for pool in (kp, vp):
        junk = torch.where(torch.rand(total, page, 1, 1, generator=g) < 0.5, float("nan"), float("inf")).to(t)
        pool.copy_(torch.where(used[..., None, None].cuda(), pool, junk.cuda()))
    q = (q_scale * torch.randn((len(lens), hq, 1, d), generator=g)).to(t)
    acc = torch.rand((len(lens), hkv, table.shape[1] * page), generator=g) if weights else None
    return table, kp, vp, k64, v64, q, acc


def run_decode(svx, case, table, kp, vp, q, acc, max_len=0, scale=0.0, cache=None, **kw):
    lens, hq, hkv, d, page, ty, layout, weights = case
    cache = cache or svx.PagedCache(kp, vp)
    o = torch.full((len(lens), hq, 1, d), 7.0, dtype=TYPES[ty], device="cuda")
    lse = torch.full((len(lens), hq, 1), 7.0, device="cuda")
    out = None if acc is None else torch.full_like(acc, 7.0, device="cuda")
    cache.decode(q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), o, lse, max_len=max_len,
                 scale=scale, acc_in=None if acc is None else acc.cuda(), acc_out=out, **kw)
    assert not cache.check()
    return o, lse, out


def check_decode(case, got, want, acc):
    lens, hq, hkv, d, page, ty, layout, weights = case
    o, lse, out = got
    o64, lse64, out64, size, spread, w = want
    n = torch.tensor(lens, dtype=torch.float64).reshape(-1, 1, 1)
    c = 2 * (2.0 ** -19 * spread + 2.0 ** -15 + n * 2.0 ** -24)
    err = (o.double().cpu() - o64).abs()
    bound = o64.abs() * unit(TYPES[ty]) + c[..., None] * size + 2.0 ** -24
    assert (err <= bound).all(), f"O: {(err / bound).max():.3f} times the bound"
    fin = torch.isfinite(lse64)
    assert torch.equal(torch.isfinite(lse.cpu()), fin) and (lse.cpu()[~fin] == -np.inf).all()
    b2 = 2.0 ** -19 * spread + 2.0 ** -20 + n * 2.0 ** -24 + lse64.abs() * 2.0 ** -22
    assert ((lse.double().cpu() - lse64).abs()[fin] <= b2.expand_as(lse64)[fin]).all()
    if acc is None:
        return
    live = torch.arange(acc.shape[-1])[None, None] < n.long()
    live = live.expand(acc.shape)
    assert (out.cpu()[~live] == 7.0).all()
    cw = c.reshape(len(lens), hkv, -1).amax(-1, keepdim=True)
    e = (out.double().cpu() - out64).abs()
    assert (e[live] <= (cw * w + out64.abs() * 2.0 ** -22)[live]).all()


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"len{c[0] if len(c[0]) < 9 else len(c[0])}-h{c[1]}-{c[2]}-d{c[3]}-p{c[4]}-{c[5]}-{c[6]}")
def test_decode(svx, case):
    table, kp, vp, k64, v64, q, acc = decode_inputs(case)
    got = run_decode(svx, case, table, kp, vp, q, acc)
    check_decode(case, got, decode64(q, k64, v64, table, case[0], case[3] ** -0.5, acc), acc)


@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("d,longest", [(128, 512), (128, 513), (64, 1024), (64, 1025)])
def test_decode_short_items_whole_and_split(svx, d, longest, hkv):
    """Items of 32 chunks stay in one CTA, one slot more and they are split; 8 heads of 20 requests are too many for it."""
    g = np.random.default_rng(longest + hkv)
    lens = (longest, 0, 1, *(int(x) for x in g.integers(0, longest + 1, 17)))
    case = (lens, 20 * hkv, hkv, d, 16, "bf16", "token", False)  # 20 query heads a KV head: two blocks
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=9)
    got = run_decode(svx, case, table, kp, vp, q, acc, max_len=longest)
    check_decode(case, got, decode64(q, k64, v64, table, case[0], d ** -0.5, acc), acc)


@pytest.mark.parametrize("q_scale", [0.0, 20.0])
def test_decode_flat_and_peaked(svx, q_scale):
    """Equal scores (the mean of V), and scores that leap: the running reference moves many times."""
    case = ((1500, 40), 6, 2, 128, 16, "fp16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=4, q_scale=q_scale)
    got = run_decode(svx, case, table, kp, vp, q, acc, scale=0.125)
    check_decode(case, got, decode64(q, k64, v64, table, case[0], 0.125, acc), acc)


def test_decode_rising_scores_and_tiny_weights(svx):
    """Keys along q, growing with the slot: every chunk raises the reference; and one slot that outweighs a long tail
    of slots whose weights lie below fp16's normal range."""
    case = ((4000,), 2, 1, 64, 16, "fp16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=5)
    for kind in ("rising", "tail"):
        s = torch.arange(4000) * 0.01 if kind == "rising" else torch.where(torch.arange(4000) == 7, 10.5, 0.0)
        q = torch.zeros_like(q)
        q[..., 0] = 8.0
        for t in range(4000):
            k64[int(table[0, t // 16]), t % 16] = 0
            k64[int(table[0, t // 16]), t % 16, :, 0] = s[t]
        good = torch.isfinite(kp)
        kp.copy_(torch.where(good, k64.cuda(), kp))
        got = run_decode(svx, case, table, kp, vp, q, acc)
        check_decode(case, got, decode64(q, k64, v64, table, case[0], 0.125, acc), acc)


def test_decode_rows_whose_scores_are_all_minus_infinity(svx):
    """q k = -inf for one query head at every slot: that row is empty (O = 0, LSE = -inf, no weight); the other is not."""
    case = ((37,), 2, 1, 64, 16, "bf16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=6)
    kp[..., 0] = torch.where(torch.isfinite(kp[..., 0]), 3.0e38, kp[..., 0].float()).to(kp.dtype)
    q[:] = 0
    q[0, 0, 0, 0] = -3.0e38
    o, lse, out = run_decode(svx, case, table, kp, vp, q, acc)
    assert (o[0, 0] == 0).all() and lse[0, 0] == -np.inf
    assert abs(float(lse[0, 1]) - np.log(37)) < 1e-5
    assert torch.allclose(out[0, 0, :37].cpu(), acc[0, 0, :37] + 1 / 37, atol=1e-6)


def test_decode_in_place_weights_and_bounded_length(svx):
    case = ((40, 700), 8, 2, 128, 16, "bf16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=7, extra=300)  # the table is far wider than the bound
    a = run_decode(svx, case, table, kp, vp, q, acc)
    b = run_decode(svx, case, table, kp, vp, q, acc, max_len=700)
    live = torch.arange(acc.shape[-1], device="cuda")[None, None] < torch.tensor([40, 700], device="cuda")[:, None, None]
    live = live.expand(acc.shape)
    want = decode64(q, k64, v64, table, case[0], case[3] ** -0.5, acc)
    check_decode(case, a, want, acc)
    check_decode(case, b, want, acc)
    buf = acc.cuda()
    cache = svx.PagedCache(kp, vp)
    o, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    cache.decode(q.cuda(), table.cuda(), torch.tensor([40, 700], dtype=torch.int32, device="cuda"), o, lse, acc_in=buf,
                 acc_out=buf)
    assert torch.equal(buf[live], a[2][live]) and torch.equal(buf[~live].cpu(), acc.cuda()[~live].cpu())
    assert torch.equal(o, a[0]) and torch.equal(lse, a[1])


def test_decode_is_deterministic_and_counts_lengths_out_of_bounds(svx):
    case = ((3000, 17, 900), 12, 3, 64, 16, "bf16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=8)
    a = run_decode(svx, case, table, kp, vp, q, acc)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, run_decode(svx, case, table, kp, vp, q, acc)))
    cache = svx.PagedCache(kp, vp)
    o, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    # beyond the bound: clamped to it and reported; below zero: an empty row and reported
    for lens, same in (((3000, -5, 900), 0), ((3000, 17, 901), 0)):
        cache.decode(q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), o, lse,
                     max_len=900 if lens[2] > 900 else 0)
        assert cache.check() and not cache.check()
    # a page that the pool does not have: reported, the other requests are right
    bad = table.clone()
    bad[1, 0] = total = kp.shape[0]
    cache.decode(q.cuda(), bad.cuda(), torch.tensor(case[0], dtype=torch.int32, device="cuda"), o, lse)
    assert cache.check() and total > 0
    assert torch.equal(o[0], a[0][0]) and torch.equal(o[2], a[0][2])


# ------------------------------------------------------------------ evict

EVICT = [  # lens, hkv, d, page, type, budget, sink, recent
    ((1,), 1, 64, 1, "bf16", 1, 0, 0),
    ((0, 1, 2, 3), 2, 128, 2, "bf16", 2, 1, 1),
    ((777, 512, 100, 0), 3, 64, 24, "fp16", 512, 4, 100),
    ((2112, 2048, 2049), 2, 128, 64, "bf16", 2048, 4, 256),
    ((1000,), 1, 128, 7, "bf16", 1, 0, 1),                  # all but one go
    ((5000, 4100), 1, 64, 16, "bf16", 2500, 0, 2500),       # every kept slot protected, or none beside them
    ((40000, 33000), 1, 64, 128, "fp16", 9000, 3, 77),      # a cluster of CTAs to a row
    ((12345,), 2, 64, 16, "bf16", 12000, 0, 0),
]


def evict_inputs(case, kind, seed=0):
    lens, hkv, d, page, ty, budget, sink, recent = case
    g = torch.Generator().manual_seed(seed)
    t = TYPES[ty]
    table, total = make_table(g, lens, page, extra=1)
    kp, vp = (torch.randn((total, page, hkv, d), generator=g).to(t).cuda() for _ in range(2))
    B, room = len(lens), table.shape[1] * page
    if kind == "weights":
        acc = torch.rand((B, hkv, room), generator=g) ** 6
    elif kind == "ties":
        acc = torch.randint(0, 3, (B, hkv, room), generator=g).float()
    else:  # signs, zeros of both signs, infinities and NaN
        acc = torch.randn((B, hkv, room), generator=g)
        pick = torch.rand((B, hkv, room), generator=g)
        for lo, v in ((0.0, float("nan")), (0.1, float("inf")), (0.2, -float("inf")), (0.3, 0.0), (0.4, -0.0)):
            acc = torch.where((pick >= lo) & (pick < lo + 0.1), torch.tensor(v), acc)
    pos = torch.stack([torch.stack([torch.randperm(2 * room, generator=g)[:room] for _ in range(hkv)]) for _ in range(B)]).to(torch.int32)
    nxt = torch.full((B,), 2 * room, dtype=torch.int32)
    return table, kp, vp, acc, pos, nxt


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["weights", "ties", "wild"])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(svx, case, kind, in_place):
    lens, hkv, d, page, ty, budget, sink, recent = case
    table, kp, vp, acc, pos, nxt = evict_inputs(case, kind)
    B = len(lens)
    k0, v0 = kp.cpu().clone(), vp.cpu().clone()
    cache = svx.PagedCache(kp, vp)
    a, p, ln = acc.cuda(), pos.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ao, po, lo = (a, p, ln) if in_place else (torch.full_like(a, 7.0), torch.full_like(p, 7), torch.full_like(ln, 7))
    cache.evict(table.cuda(), ln, budget, sink, recent, nxt.cuda(), a, p, ao, po, lo)
    assert not cache.check()
    assert lo.tolist() == [min(n, budget) for n in lens]
    want_a = acc.clone() if in_place else torch.full_like(acc, 7.0)
    want_p = pos.clone() if in_place else torch.full_like(pos, 7)
    k1, v1 = k0.clone(), v0.clone()
    for b, n in enumerate(lens):
        for h in range(hkv):
            order = evict64(acc[b, h].numpy(), pos[b, h].numpy(), n, int(nxt[b]), budget, sink, recent)
            want_a[b, h, :len(order)], want_p[b, h, :len(order)] = acc[b, h][order], pos[b, h][order]
            for to, fro in enumerate(order):
                if to != fro:
                    pt, pf = int(table[b, to // page]), int(table[b, fro // page])
                    k1[pt, to % page, h], v1[pt, to % page, h] = k0[pf, fro % page, h], v0[pf, fro % page, h]
    assert torch.equal(po.cpu(), want_p)
    assert torch.equal(torch.nan_to_num(ao.cpu(), nan=1e30), torch.nan_to_num(want_a, nan=1e30))
    assert torch.equal(kp.cpu(), k1) and torch.equal(vp.cpu(), v1)


def test_evict_bad_page_is_reported_and_left_out(svx):
    case = ((200, 200), 1, 64, 16, "bf16", 100, 0, 0)
    table, kp, vp, acc, pos, nxt = evict_inputs(case, "weights")
    k0 = kp.clone()
    bad = table.clone()
    bad[0, :] = -1
    cache = svx.PagedCache(kp, vp)
    ln = torch.tensor(case[0], dtype=torch.int32, device="cuda")
    ao, po, lo = torch.empty_like(acc, device="cuda"), torch.empty_like(pos, device="cuda"), torch.empty_like(ln)
    cache.evict(bad.cuda(), ln, 100, 0, 0, nxt.cuda(), acc.cuda(), pos.cuda(), ao, po, lo)
    assert cache.check() and not cache.check()
    mine = table[0, :13].long().cuda()
    assert torch.equal(kp[mine], k0[mine])  # the pages that the broken table no longer names
