"""One-token attention behind shared prefixes on the GPU against a plain 64-bit implementation (bounds: attention_reference.near).

With up to 128 rows (query heads of a KV head times requests) a softmax weight enters the product with V in two 16-bit pieces, within 2^-15 of
itself with its exponential and its sum; with more it is rounded to the inputs' type once, by half a step."""
import pytest
import torch

from attention_reference import attend64, near, slots_of

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def p_error(rows, ty):
    return 2.0 ** -15 + (torch.finfo(TYPES[ty]).eps / 2 if rows > 128 else 0.0)


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def make(groups, before, behind, prefix, own, hq, hkv, d, page, ty, layout="token", seed=0, extra=1):
    """groups: requests of each prefix; before, behind: requests without one; own: each request's length."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[ty]
    batch = before + sum(groups) + behind
    own = [own[i % len(own)] for i in range(batch)]
    need = [-(-n // page) for n in list(prefix) + own]
    order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    far = torch.full((len(prefix), max(need[:len(prefix)] + [1]) + extra), -1, dtype=torch.int32)
    table = torch.full((batch, max(need[len(prefix):] + [1]) + extra), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        row = far[i] if i < len(prefix) else table[i - len(prefix)]
        row[:n] = order[at:at + n]
        at += n
    shape = (len(order), page, hkv, d) if layout == "token" else (len(order), hkv, page, d)
    k, v = ((torch.randn(shape, generator=g)).to(t).cuda() for _ in range(2))
    if layout == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    # what lies behind the lengths is not a number
    live = torch.zeros((len(order), page), dtype=torch.bool)
    for i, n in enumerate(list(prefix) + own):
        row = far[i] if i < len(prefix) else table[i - len(prefix)]
        s = torch.arange(n)
        live[row[s // page].long(), s % page] = True
    k[~live.cuda()], v[~live.cuda()] = float("nan"), float("nan")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=(2 * torch.randn((batch, hq, 1, d), generator=g)).to(t).cuda(), k=k, v=v, far=far.cuda(), table=table.cuda(),
                prefix_lens=ints(list(prefix)), lens=ints(own),
                first=ints([before + sum(groups[:i]) for i in range(len(groups) + 1)]),
                o=torch.full((batch, hq, 1, d), 7.0, dtype=t, device="cuda"), lse=torch.full((batch, hq, 1), 7.0, device="cuda"))


def run(c, s, **kw):
    c.decode_shared(s["q"], s["far"], s["prefix_lens"], s["first"], s["table"], s["lens"], s["o"], s["lse"], **kw)


def check(s, ty, scale=None, first=None, prefix_lens=None, lens=None):
    batch, hq, _, d = s["q"].shape
    hkv = s["k"].shape[2]
    group = hq // hkv
    first = s["first"].tolist() if first is None else first
    prefix_lens = s["prefix_lens"].tolist() if prefix_lens is None else prefix_lens
    lens = s["lens"].tolist() if lens is None else lens
    rows = [[slots_of(s[x], s["far"][p], n) for x in "kv"] for p, n in enumerate(prefix_lens)]
    for b in range(batch):
        mine = [slots_of(s[x], s["table"][b], lens[b]) for x in "kv"]
        for p in range(len(prefix_lens)):
            if first[p] <= b < first[p + 1]:
                mine = [torch.cat((rows[p][i], mine[i])) for i in range(2)]
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            want = attend64(s["q"][b, heads, 0], mine[0][:, h], mine[1][:, h], scale or d ** -0.5)
            near(s["o"][b, heads, 0], s["lse"][b, heads, 0], want, p_error(batch * group, ty), len(mine[0]))


CASES = [  # groups, before, behind, prefix, own, hq, hkv, d, page, type, layout
    ((1,), 0, 0, (1,), (0,), 1, 1, 64, 1, "bf16", "token"),
    ((1,), 0, 0, (0,), (0,), 4, 2, 128, 16, "bf16", "token"),
    ((4,), 0, 0, (512,), (3, 0, 40), 4, 1, 64, 16, "bf16", "token"),
    ((2, 0, 3), 1, 2, (200, 50, 129), (0, 1, 17, 200), 8, 2, 128, 16, "fp16", "token"),
    ((5, 1, 7), 0, 2, (777, 5000, 2999), (0, 300, 1, 77), 28, 4, 128, 24, "fp16", "head"),
    ((16,), 0, 0, (1000,), (64, 63, 65), 32, 8, 128, 64, "bf16", "token"),          # 64 rows to a KV head
    ((33,), 0, 1, (1025,), (5, 130), 8, 2, 64, 100, "bf16", "head"),                # 132 rows
    ((70, 3), 0, 0, (640, 6000), (10, 0, 1), 8, 1, 128, 32, "bf16", "token"),        # 560 rows, 24 rows
    ((200, 56), 0, 0, (300, 128), (0, 2), 2, 1, 64, 8, "fp16", "token"),             # the most requests
    ((3,), 2, 1, (90,), (450, 90), 17, 1, 128, 16, "bf16", "token"),                 # 17 heads to a KV head: blocks of 16 and 1
    ((2,), 0, 0, (40000,), (100,), 8, 1, 128, 16, "bf16", "token"),                  # one prefix over many CTAs
    ((1,) * 100, 0, 0, tuple(range(100)), (3,), 2, 2, 64, 16, "bf16", "token"),      # many prefixes of one request
    ((40,), 0, 0, (9000,), (9000, 1, 0), 12, 3, 64, 128, "fp16", "token"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_shared(svx, case):
    groups, before, behind, prefix, own, hq, hkv, d, page, ty, layout = case
    s = make(groups, before, behind, prefix, own, hq, hkv, d, page, ty, layout)
    c = svx.PagedCache(s["k"], s["v"])
    run(c, s)
    check(s, ty)
    assert not c.check()
    want_o, want_lse = s["o"].clone(), s["lse"].clone()
    s["o"].fill_(3)
    run(c, s, max_prefix=max(max(prefix), 1), max_len=max(max(own), 1))  # bounds: the same but for the order of sums
    check(s, ty)
    for _ in range(3):
        run(c, s)
        assert torch.equal(s["o"], want_o) and torch.equal(s["lse"], want_lse)


def test_as_decode_over_joined_tables(svx):
    """Prefixes that end with a page: the same slots as one sequence of decode."""
    s = make((3, 2), 0, 1, (320, 64), (10, 55, 1), 16, 4, 128, 32, "bf16")
    c = svx.PagedCache(s["k"], s["v"])
    run(c, s)
    both, lens = torch.full((6, 14), -1, dtype=torch.int32, device="cuda"), s["lens"].clone()
    for b in range(6):
        p = 0 if b < 3 else 1 if b < 5 else None
        n = 0 if p is None else (320, 64)[p] // 32
        if n:
            both[b, :n] = s["far"][p, :n]
        both[b, n:n + s["table"].shape[1]] = s["table"][b][:14 - n]
        lens[b] += n * 32
    o, lse = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
    c.decode(s["q"], both, lens, o, lse)
    assert (o.float() - s["o"].float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert (lse - s["lse"]).abs().max() < 1e-5
    check(s, "bf16")


@pytest.mark.parametrize("batch", [3, 40])
def test_sharp_softmax_and_scales(svx, batch):
    s = make((batch,), 0, 0, (1500,), (200, 3), 4, 1, 128, 16, "fp16", seed=2)
    t = torch.arange(1500)
    where = (s["far"][0].cpu()[t // 16].long().cuda(), (t % 16).cuda())
    for sign in (1, -1):
        s["k"][where[0], where[1], 0, 0] = (sign * torch.linspace(-12, 12, 1500)).to(s["k"].dtype).cuda()
        c = svx.PagedCache(s["k"], s["v"])
        run(c, s, scale=1.0)
        check(s, "fp16", scale=1.0)


@pytest.mark.parametrize("batch", [2, 60])
def test_what_is_out_of_bounds_on_the_device_is_clamped_and_reported(svx, batch):
    s = make((batch,), 1, 1, (100,), (20, 0, 33), 8, 2, 64, 16, "bf16", seed=3, extra=0)
    c = svx.PagedCache(s["k"], s["v"])
    lens, far = s["lens"].tolist(), s["prefix_lens"].tolist()
    run(c, s)
    assert not c.check()
    good = s["o"].clone()
    s["lens"][0] = -5
    run(c, s)
    check(s, "bf16", lens=[0] + lens[1:])
    assert c.check()
    s["lens"][0] = lens[0]
    s["prefix_lens"][0] = -1
    run(c, s)
    check(s, "bf16", prefix_lens=[0], lens=lens)
    assert c.check()
    s["prefix_lens"][0] = far[0]
    first = s["first"].tolist()
    for bad, now in (([-3, first[1]], [0, first[1]]), ([1, 1000], [1, batch + 2]), ([5, 1], [5, 5])):
        s["first"].copy_(torch.tensor(bad))
        if now[0] > batch + 2:
            continue
        run(c, s)
        check(s, "bf16", first=[min(x, batch + 2) for x in now])
        assert c.check()
    s["first"].copy_(torch.tensor(first))
    table = s["far"].clone()
    s["far"][0, 1] = 1 << 30  # a page that is not there: its slots are left out, nothing is read
    run(c, s)
    assert c.check()
    s["far"].copy_(table)
    run(c, s)
    assert torch.equal(s["o"], good) and not c.check()


def test_overlapping_ranges_do_not_fall(svx):
    """first falls: a prefix begins where those before it have begun, at least."""
    s = make((3, 3, 2), 0, 0, (50, 60, 70), (5,), 4, 2, 64, 16, "bf16", seed=4)
    c = svx.PagedCache(s["k"], s["v"])
    s["first"].copy_(torch.tensor([0, 5, 2, 8]))
    run(c, s)
    check(s, "bf16", first=[0, 5, 5, 8])
    assert c.check()


@pytest.mark.parametrize("batch", [4, 50])
def test_graph_replayed_as_lengths_and_groups_change(svx, batch):
    s = make((batch, 1), 0, 0, (700, 300), (60, 0, 31), 8, 2, 128, 16, "bf16", seed=5)
    c = svx.PagedCache(s["k"], s["v"])
    run(c, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, s)
    most = s["lens"].clone()
    for far, own, first in (((700, 0), 1, (0, batch, batch + 1)), ((1, 300), 0, (0, 1, batch + 1)), ((699, 128), 1, (1, 2, 3))):
        s["prefix_lens"].copy_(torch.tensor(far))
        s["lens"].copy_(most * own)
        s["first"].copy_(torch.tensor(first))
        s["o"].fill_(3)
        graph.replay()
        check(s, "bf16")
    assert not c.check()


def test_two_calls_at_once(svx):
    s = make((20,), 0, 0, (3000,), (50, 7), 8, 2, 128, 16, "bf16", seed=6)
    c = svx.PagedCache(s["k"], s["v"])
    run(c, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [{**s, "o": torch.zeros_like(s["o"]), "lse": torch.zeros_like(s["lse"])} for _ in streams]
    for _ in range(10):
        for x, st in zip(outs, streams):
            run(c, x, stream=st)
    torch.cuda.synchronize()
    for x in outs:
        assert torch.equal(x["o"], s["o"]) and torch.equal(x["lse"], s["lse"])


def test_refusals(svx):
    s = make((3,), 0, 0, (40,), (5,), 4, 2, 64, 16, "bf16")
    c = svx.PagedCache(s["k"], s["v"])
    bad = [dict(q=s["q"].half()), dict(q=s["q"][..., 0, :]), dict(far=s["far"].long()), dict(far=s["far"][0]),
           dict(prefix_lens=s["prefix_lens"].repeat(2)), dict(first=s["first"][:1]), dict(first=s["first"].cpu()),
           dict(table=s["table"][:2]), dict(lens=s["lens"][:2]), dict(o=s["o"].float()), dict(o=s["q"]), dict(lse=s["lse"].half()),
           dict(q=s["q"][:, :3].contiguous(), o=s["o"][:, :3].contiguous(), lse=s["lse"][:, :3].contiguous()),
           dict(far=s["far"][:0], prefix_lens=s["prefix_lens"][:0], first=s["first"][:1])]
    for change in bad:
        with pytest.raises(svx.SvxError):
            run(c, {**s, **change})
    for kw in (dict(scale=-1.0), dict(max_prefix=-1), dict(max_prefix=10 ** 6), dict(max_len=10 ** 6),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(svx.SvxError):
            run(c, s, **kw)
    inside = s["k"].view(-1)[:s["o"].numel()].view(s["o"].shape)
    with pytest.raises(svx.SvxError):
        run(c, {**s, "o": inside})
    with pytest.raises(svx.SvxError):
        run(c, s, workspace=s["v"])
