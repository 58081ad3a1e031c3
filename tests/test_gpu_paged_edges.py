"""Edges of the paged-cache operators on the GPU: calls that the header allows and whose results hang on one detail.

Bounds are derived at each test; u = torch.finfo(type).eps / 2 is a rounding to the output type.
"""
import math

import pytest
import torch

from paged_reference import decode64, evict64, heads64
from test_gpu_paged import HEADS, check_decode, decode_inputs, heads_inputs, heads_reference, make_table, near, run_decode

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ heads


def pair_terms(y, pos, inv_freq, neighbours):
    """|y_a cos t| + |y_b sin t| and |y_b cos t| + |y_a sin t| at their places: the size that a rotated value's error goes by."""
    half = len(inv_freq)
    ang = torch.as_tensor(pos, dtype=torch.float64)[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(ang).abs()[:, None], torch.sin(ang).abs()[:, None]
    out = y.abs().clone()
    ia = torch.arange(half) * 2 if neighbours else torch.arange(half)
    ib = ia + (1 if neighbours else half)
    a, b = y[..., ia].abs(), y[..., ib].abs()
    out[..., ia], out[..., ib] = a * c + b * s, b * c + a * s
    return out


@pytest.mark.parametrize("zero", ["first", "second", "none"])
@pytest.mark.parametrize("neighbours", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("d,ty", [(128, "bf16"), (128, "fp16"), (64, "fp16"), (64, "bf16")])
def test_small_angles_keep_their_sine(svx, d, ty, neighbours, zero):
    """A pair with one member zero shows sine and cosine themselves, down to angles of 1e-7: each output is within its own rounding.
    In fp32 (u' = 2^-24): angle, sine and cosine within 4 u' relative, two products and a sum 2 u', the scale 1 u': under 2^-20 of
    |y_a cos t| + |y_b sin t|, and a sum rounded to the type.  (The angle's phase is off by 2^-55 |pos| turns at most: nothing beside.)"""
    t, n = TYPES[ty], 600
    g = torch.Generator().manual_seed(21)
    x = torch.randn((1, n, 2, d), generator=g).to(t)
    first = torch.zeros(d, dtype=torch.bool)
    if neighbours:
        first[0::2] = True
    else:
        first[:d // 2] = True
    if zero != "none":
        x[..., first if zero == "first" else ~first] = 0
    pos = torch.cat([torch.arange(-100, 300), torch.randint(-2 ** 20, 2 ** 20, (n - 400,), generator=g)]).to(torch.int32)[None]
    inv = [1e6 ** (-2.0 * i / d) for i in range(d // 2)]
    inv[1], inv[3] = 3e-7, 1.0 / 65536  # (positions times 2^-16 reach the quadrants' borders to within an ulp)
    inv[5] = math.pi / 4
    qo, ko = torch.empty((1, 1, n, d), dtype=t, device="cuda"), torch.empty((1, n, 1, d), dtype=t, device="cuda")
    xc = x.cuda()
    svx.qk_norm_rope(xc[:, :, :1], xc[:, :, 1:], None, pos.cuda(), svx.Rope(d, inv_freq=inv, neighbours=neighbours), qo, ko, eps=None)
    for got, h in ((qo[0].transpose(0, 1), 0), (ko[0], 1)):
        z, _ = heads64(x[0, :, h:h + 1], None, None, pos[0], inv, neighbours)
        size = pair_terms(x[0, :, h:h + 1].double(), pos[0], inv, neighbours)
        # the reference's own angle: 64-bit products of up to 2^20 are off by 2^-33 radians at most
        bound = z.abs() * torch.finfo(t).eps / 2 + size * 2.0 ** -20 + x[0, :, h:h + 1].double().abs().amax() * 2.0 ** -33 \
            + torch.finfo(t).tiny * torch.finfo(t).eps
        err = (got.double().cpu() - z).abs()
        assert (err <= bound).all(), f"{float((err / bound).max()):.2f} times the bound at {int((err > bound).sum())} elements"


# ------------------------------------------------------------------ one-token attention


@pytest.mark.parametrize("which", ["k", "v"])
def test_decode_refuses_a_workspace_in_the_pools(svx, which):
    """The workspace's size needs the device's SM count, so this is seen here: a workspace that begins in a pool, ends in it, or lies
    beside it."""
    n = 4 * 16 * 2 * 64
    need = svx.ctypes.c_int64(0)
    arena = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    mine = arena[1 << 23:(1 << 23) + 2 * n].view(torch.bfloat16).view(4, 16, 2, 64)
    other = torch.zeros_like(mine)
    cache = svx.PagedCache(*((mine, other) if which == "k" else (other, mine)))
    q, o = (torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, table, lens = torch.zeros((1, 4, 1), device="cuda"), i32([[0, 1, 2]]), i32([40])
    p = svx.Pages.from_buffer_copy(cache._pages)
    p.table, p.max_pages = table.data_ptr(), 3
    assert svx.lib.svx_paged_decode_workspace(svx.ctypes.byref(p), 1, 4, 0, 0, svx.ctypes.byref(need)) == svx.OK
    size = (need.value + 255) // 256 * 256
    for at in ((1 << 23), (1 << 23) + 2 * n - 256, (1 << 23) - size + 256):
        with pytest.raises(svx.SvxError, match="overlap"):
            cache.decode(q, table, lens, o, lse, workspace=arena[at:at + size])
    for at in ((1 << 23) + 2 * n, (1 << 23) - size):
        cache.decode(q, table, lens, o, lse, workspace=arena[at:at + size])
    assert not cache.check()


# ------------------------------------------------------------------ the bounds-checked library


def test_strays_name_the_buffer_that_they_left(svx):
    """With buffers described as smaller than they are (svx_debug_clip_paged), the checked library skips what lies past the end and names the
    buffer; the other library, and the next call, do all of it."""
    checked = "bounds-checked" in svx.version()
    g = torch.Generator().manual_seed(22)
    n, hq, hkv, d, page, t = 6, 4, 2, 64, 4, torch.bfloat16
    x = torch.randn((1, n, hq + 2 * hkv, d), generator=g).to(t).cuda()
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    pos, rope, table, start = i32([list(range(n))]), svx.Rope(d), i32([[0, 1]]), i32([1])
    qo = torch.zeros((1, hq, n, d), dtype=t, device="cuda")
    ko, vo = (torch.zeros((1, n, hkv, d), dtype=t, device="cuda") for _ in range(2))
    kp, vp = (torch.zeros((2, page, hkv, d), dtype=t, device="cuda") for _ in range(2))
    cache, status = svx.PagedCache(kp, vp), i32([0])
    o, lse, lens = torch.zeros((1, hq, 1, d), dtype=t, device="cuda"), torch.zeros((1, hq, 1), device="cuda"), i32([n + 1])
    acc = torch.zeros((1, hkv, 2 * page), device="cuda")
    spos = torch.zeros((1, hkv, 2 * page), dtype=torch.int32, device="cuda")

    def dense():
        svx.qk_norm_rope(q, k, v, pos, rope, qo, ko, vo, status=status)
        return status

    def append():
        cache.append(q, k, v, pos, rope, table, start, qo)
        return cache.status

    def decode():
        cache.decode(q[:, :1].transpose(1, 2).contiguous(), table, lens, o, lse)
        return cache.status

    def evict():
        cache.evict(table, lens, 3, 0, 3, i32([8]), acc, spos.copy_(torch.arange(2 * page, device="cuda").int().expand_as(spos)), acc,
                    spos, i32([0]))
        return cache.status

    def clip(buffer, elements):
        assert svx.lib.svx_debug_clip_paged(buffer, elements) == svx.OK
    inside, outside, pool = 1 << 17, 1 << 18, 1 << 19
    cases = [(dense, 0, 3 * (hq + 2 * hkv) * d, inside), (append, 0, 3 * (hq + 2 * hkv) * d, inside), (dense, 1, 2 * hkv * d, outside),
             (append, 1, 2 * hkv * d, outside), (append, 2, page * hkv * d, pool), (decode, 2, page * hkv * d, pool), (evict, 2, page * hkv * d, pool)]
    for call, buffer, elements, bit in cases:
        word = call()
        assert int(word) == 0, call.__name__
        for y in (qo, ko, vo):
            y.zero_()
        try:
            clip(buffer, elements)
            call()
        finally:
            clip(buffer, -1)
        assert int(word) == (4 | bit if checked else 0), (call.__name__, buffer, hex(int(word)))
        word.zero_()
        if checked and buffer == 1:
            assert (qo.view(-1)[2 * hkv * d:] == 0).all() and (qo.view(-1)[:2 * hkv * d] != 0).any()
            if call is dense:
                assert (ko.view(-1)[2 * hkv * d:] == 0).all() and (vo.view(-1)[2 * hkv * d:] == 0).all() and (vo.view(-1)[:2 * hkv * d] != 0).any()
        call()
        assert int(word) == 0
    assert svx.lib.svx_debug_clip_paged(3, 0) == svx.ERR_INVALID_ARG


# ------------------------------------------------------------------ eviction: every kernel that the lengths choose

# longest, rows (requests x KV heads), d, page, evicted slots, most moves: by the longest row 256, 512 or 1024 threads of 4 to 32 keys and
# clusters of 1 to 8; with up to 64 (256 threads) or 128 (512) moves and a length of its own they are made in the selecting kernel
SELECT = [
    (1000, (2, 2), 64, 24, 41),       # 256 threads, moves in several warps, a remainder
    (1000, (1, 3), 64, 7, 9),
    (1024, (2, 1), 128, 16, 64),      # at the limits: 4 keys, 64 moves
    (1025, (2, 2), 128, 16, 65),      # one past both
    (2048, (1, 2), 128, 32, 58),
    (2049, (1, 2), 64, 32, 63),
    (2560, (2, 1), 64, 64, 33),
    (2561, (2, 1), 128, 64, 100),     # 512 threads
    (4096, (1, 2), 64, 16, 127),
    (4097, (1, 2), 128, 16, 128),
    (6144, (1, 1), 64, 100, 128),
    (6145, (1, 1), 64, 100, 129),
    (8192, (2, 1), 128, 128, 77),
    (8193, (2, 1), 128, 128, 77),     # 1024 threads
    (12289, (1, 2), 64, 128, 5000),
    (16384, (1, 1), 64, 128, 300),
    (16385, (1, 1), 64, 128, 300),    # two CTAs to a row
    (17000, (10, 8), 64, 128, 700),   # as long, but the rows fill the card: 32 keys a thread
    (70000, (5, 4), 64, 256, 900),    # four CTAs, 32 keys
    (262144, (1, 2), 64, 1024, 2000),  # the longest: eight
]


PLACES = ["apart", "weights in place", "all in place"]


@pytest.mark.parametrize("case,place", [(c, p) for c in SELECT for p in PLACES if c[0] < 16385 or p != "weights in place"],
                         ids=lambda c: c if isinstance(c, str) else f"len{c[0]}-rows{c[1][0]}x{c[1][1]}-d{c[2]}-gone{c[4]}")
def test_evict_with_every_selecting_kernel(svx, case, place):
    """Each row loses exactly `gone` slots in front, so that as many rows of K and V move; a shorter request moves fewer.  Exact."""
    longest, (B, hkv), d, page, gone = case
    g = torch.Generator().manual_seed(longest)
    lens = [longest - (11 * b if b else 0) for b in range(B)]
    budget = longest - gone
    table, total = make_table(g, lens, page)
    kp, vp = (torch.randn((total, page, hkv, d), generator=g).to(torch.float16).cuda() for _ in range(2))
    k0, v0 = kp.clone(), vp.clone()
    room = table.shape[1] * page
    acc = 1 + torch.rand((B, hkv, room), generator=g)
    pos = torch.stack([torch.stack([torch.randperm(room, generator=g) for _ in range(hkv)]) for _ in range(B)]).to(torch.int32)
    recent = budget // 8
    for b, n in enumerate(lens):
        for h in range(hkv):  # the lightest lie in front, and none of them is protected by its position
            low = torch.randperm(budget, generator=g)[:gone]
            acc[b, h, low] = torch.rand(gone, generator=g)
            late = pos[b, h, low] >= room - recent
            pos[b, h, low[late]] = 5
    nxt = i32([room] * B)
    a, p, ln = acc.cuda(), pos.cuda(), i32(lens)
    ao, po = (a, p) if "place" in place else (torch.full_like(a, 7.0), torch.full_like(p, 7))
    lo = ln if place == "all in place" else torch.full_like(ln, 7)
    cache = svx.PagedCache(kp, vp)
    cache.evict(table.cuda(), ln, budget, 0, recent, nxt, a, p, ao, po, lo, max_len=longest)
    assert not cache.check() and lo.tolist() == [min(n, budget) for n in lens]
    td = table.cuda().long()
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(hkv):
            order = torch.tensor(evict64(acc[b, h].numpy(), pos[b, h].numpy(), n, room, budget, 0, recent))
            assert int((order != torch.arange(m)).sum()) == n - m
            assert torch.equal(ao[b, h, :m].cpu(), acc[b, h][order]) and torch.equal(po[b, h, :m].cpu(), pos[b, h][order])
            to, fro = torch.arange(m).cuda(), order.cuda()
            for pool, old in ((kp, k0), (vp, v0)):
                assert torch.equal(pool[td[b, to // page], to % page, h], old[td[b, fro // page], fro % page, h])
            rest = torch.arange(m, n).cuda()  # what lies behind stays
            assert torch.equal(kp[td[b, rest // page], rest % page, h], k0[td[b, rest // page], rest % page, h])
            if place == "apart":
                assert (ao[b, h, m:] == 7.0).all() and (po[b, h, m:] == 7).all()
            else:
                assert torch.equal(ao[b, h, m:].cpu(), acc[b, h, m:]) and torch.equal(po[b, h, m:].cpu(), pos[b, h, m:])


# ------------------------------------------------------------------ what is reported, and what it leaves right


@pytest.mark.parametrize("case", HEADS, ids=str)
def test_heads_with_a_status_word_report_nothing(svx, case):
    """The dense form with a status word (without one the checked library has nowhere to report a stray): clear, and the values right."""
    b, n, hq, hkv, d, rot, nb, norm, ty, scale = case
    qkv, pos, wq, wk, inv = heads_inputs(case, seed=23)
    t, status, x = TYPES[ty], i32([0]), qkv.cuda()
    qo, ko, vo = (torch.full(s, 7.0, dtype=t, device="cuda") for s in ((b, hq, n, d), (b, n, hkv, d), (b, n, hkv, d)))
    cu = lambda w: None if w is None else w.cuda()  # noqa: E731
    svx.qk_norm_rope(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos.cuda(), svx.Rope(rot, inv_freq=inv, neighbours=nb, scale=scale),
                     qo, ko, vo, q_norm=cu(wq), k_norm=cu(wk), eps=1e-6 if norm else None, status=status)
    assert int(status) == 0
    q, qs, k, ks, v = heads_reference(case, qkv, pos, wq, wk, inv)
    near(qo.transpose(1, 2), q, qs, t)
    near(ko, k, ks, t)
    assert torch.equal(vo.cpu(), v)


def test_lengths_out_of_bounds_are_clamped(svx):
    """As the header says of what lies on the device: a negative length counts as none, one above max_len as max_len; other requests'
    rows are those of a call without the fault, bit for bit."""
    case = ((3000, 17, 900), 12, 3, 64, 16, "bf16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=24)
    for lens, right, max_len in (((3000, -5, 900), (3000, 0, 900), 0), ((3000, -2 ** 31, 900), (3000, 0, 900), 0), ((901, 17, 900), (900, 17, 900), 900),
                                 ((2 ** 31 - 1, 17, 900), (900, 17, 900), 900)):
        cache = svx.PagedCache(kp, vp)
        want = run_decode(svx, (right, *case[1:]), table, kp, vp, q, acc, max_len=max_len)
        check_decode((right, *case[1:]), want, decode64(q, k64, v64, table, right, case[3] ** -0.5, acc), acc)
        o, lse, out = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0), torch.full_like(want[2], 7.0)
        cache.decode(q.cuda(), table.cuda(), i32(lens), o, lse, max_len=max_len, acc_in=acc.cuda(), acc_out=out)
        assert cache.check() and not cache.check()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(out, want[2])
        if right[1] == 0:
            assert (o[1] == 0).all() and (lse[1] == -float("inf")).all() and (out[1] == 7.0).all()


def test_values_that_are_not_finite_stay_with_their_request(svx):
    """K and V below a length have to be finite; one that is not spoils its own request and KV head, and no other."""
    case = ((70, 700, 300), 8, 2, 128, 16, "bf16", "token", True)
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=25)
    good = run_decode(svx, case, table, kp, vp, q, acc)
    for pool in (kp, vp):
        old = pool.clone()
        for value in (float("inf"), float("nan"), -float("inf")):
            pool.copy_(old)
            pool[int(table[1, 200 // 16]), 200 % 16, 1, 3] = value
            o, lse, out = run_decode(svx, case, table, kp, vp, q, acc)
            assert math.isinf(value) and pool is kp or not torch.isfinite(o[1, 4:]).all()  # (a score of -inf is a weight of 0)
            assert torch.equal(o[1, :4], good[0][1, :4]) and torch.equal(lse[1, :4], good[1][1, :4]) and torch.equal(out[1, 0], good[2][1, 0])
            for b in (0, 2):
                assert all(torch.equal(x[b], y[b]) for x, y in zip((o, lse, out), good))
        pool.copy_(old)


def test_no_room_for_a_workspace_is_an_out_of_memory_error(svx):
    """Scores of 4096 heads over 2^25 slots are 512 GiB: torch's allocator refuses, as it does in torch's own calls, and the next call runs."""
    page, room = 1 << 15, 1 << 25
    kp, vp = (torch.zeros((1, page, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache, table = svx.PagedCache(kp, vp), torch.zeros((1, room // page), dtype=torch.int32, device="cuda")
    q, lens = torch.zeros((1, 4096, 1, 64), dtype=torch.bfloat16, device="cuda"), i32([3])
    o, lse, acc = torch.full_like(q, 7.0), torch.empty((1, 4096, 1), device="cuda"), torch.zeros((1, 1, room), device="cuda")
    with pytest.raises(torch.cuda.OutOfMemoryError):
        cache.decode(q, table, lens, o, lse, acc_in=acc, acc_out=acc)
    cache.decode(q, table, lens, o, lse, max_len=64, acc_in=acc, acc_out=acc)
    assert not cache.check() and (o == 0).all()
    assert torch.allclose(acc[0, 0, :3], torch.full((3,), 4096 / 3, device="cuda"), rtol=1e-4) and (acc[0, 0, 3:] == 0).all()


@pytest.mark.parametrize("page", [77, 100, 1000, 4097, 65535, 99991, (1 << 20) + 7])
def test_slots_find_their_page_up_to_the_last(svx, page):
    """The division by page_size that the kernels make by multiplication, as the host sets it up: single tokens at slots around page borders up
    to 2^31 - 1, in a table whose only page is the right one."""
    pages = (2 ** 31 - 1) // page
    kp, vp = (torch.zeros((1, page, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache, rope = svx.PagedCache(kp, vp), svx.Rope(64)
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(page)
    slots = {0, page - 1, page, pages * page - 1, pages * page - page}
    for p in torch.randint(0, pages, (12,), generator=g).tolist():
        slots |= {p * page, p * page + page - 1, p * page + page // 2}
    qo = torch.empty((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    for i, slot in enumerate(sorted(slots)):
        table[0, slot // page] = 0
        x = torch.full((1, 1, 3, 64), float(i + 1), dtype=torch.bfloat16, device="cuda")
        cache.append(x[:, :, :1], x[:, :, 1:2], x[:, :, 2:], i32([[0]]), rope, table, i32([slot]), qo, eps=None)
        assert not cache.check(), slot
        assert (vp[0, slot % page] == i + 1).all() and (kp[0, slot % page] == i + 1).all(), slot
        table[0, slot // page] = -1
        vp[0, slot % page] = 0
    assert not vp.any()  # nothing went anywhere else
