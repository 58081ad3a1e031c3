"""Edges of attention to an encoder's states and behind shared prefixes on the GPU: layouts, alignment, far offsets, every kernel that the
rules choose, the bounds-checked library's hook, and a decoder layer that uses them together with the residual stream.  Bounds:
attention_reference.near, with the roundings of test_gpu_cross.py and test_gpu_shared.py; test_gpu_residual.py for the stream."""
import ctypes
import math
import os

import pytest
import torch

from attention_reference import attend64, near, slots_of

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CHECKED = os.environ.get("SVX_LIBRARY") == "checked"


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def p_error(rows, t):
    return 2.0 ** -15 + (torch.finfo(t).eps / 2 if rows > 128 else 0.0)


def check_cross(q, k, v, o, lse, seen=None, heads=None):
    b, hq, n, d = q.shape
    group = hq // k.shape[2]
    for i in range(b):
        at = torch.arange(k.shape[1], device="cuda") if seen is None else seen[i].nonzero()[:, 0]
        for h in range(k.shape[2]) if heads is None else heads:
            x = slice(h * group, (h + 1) * group)
            want = attend64(q[i, x].reshape(-1, d), k[i, at, h], v[i, at, h], d ** -0.5)
            near(o[i, x].reshape(-1, d), lse[i, x].reshape(-1), want, p_error(group * n, q.dtype), len(at))


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n, hq, hkv", [(3, 4, 1), (5, 10, 1), (20, 4, 2), (32, 4, 1), (33, 4, 1), (100, 3, 1), (64, 8, 2), (300, 2, 2)])
def test_rows_around_the_limits_of_the_kernels(svx, n, hq, hkv, d, ty):
    """12 to 300 rows: one block of 16, one row tile, two, more than two; whole tokens to a row tile and not."""
    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(TYPES[ty])  # noqa: E731
    for states in (127, 128, 385, 2000):
        q, k, v = 2 * r(2, hq, n, d), r(2, states, hkv, d), r(2, states, hkv, d)
        o, lse = torch.full_like(q, 7.0), torch.full((2, hq, n), 7.0, device="cuda")
        svx.cross_attn(q, k, v, o, lse)
        check_cross(q, k, v, o, lse)


@pytest.mark.parametrize("n", [2, 50, 150])
def test_addresses_on_the_16_byte_grid_only(svx, n):
    """Every tensor begins 16 bytes behind a 256-byte boundary, with strides that are odd multiples of 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(7)

    def odd(*shape):
        rows = math.prod(shape[:-1])
        wide = torch.randn(rows * (shape[-1] + 8) + 8, generator=g, device="cuda").half()
        return wide[8:].view(rows, shape[-1] + 8)[:, :shape[-1]].view(*shape[:-1], shape[-1])

    q, k, v, o = odd(2, n, 4, 128).transpose(1, 2), odd(2, 700, 2, 128), odd(2, 700, 2, 128), odd(2, n, 4, 128).transpose(1, 2)
    lse = torch.zeros((2, 4, n), device="cuda")
    svx.cross_attn(q, k, v, o, lse)
    check_cross(q, k, v, o, lse)


@pytest.mark.parametrize("n", [1, 40, 200])
def test_a_mask_off_the_word_grid(svx, n):
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(3, 2, n, 64), r(3, 301, 1, 64), r(3, 301, 1, 64)
    mask = (torch.rand(3 * 307 + 3, generator=g, device="cuda") < 0.5)[3:].view(3, 307)[:, :301]
    k[~mask], v[~mask] = float("nan"), float("-inf")
    o, lse = torch.zeros_like(q), torch.zeros((3, 2, n), device="cuda")
    svx.cross_attn(q, k, v, o, lse, mask=mask)
    check_cross(q, k, v, o, lse, mask)


@pytest.mark.parametrize("n", [1, 20])
def test_states_past_two_to_the_31_elements(svx, n):
    """4.6 GB of states: the last of them decide."""
    states, hkv, d = 1_110_000, 8, 128
    kv = torch.zeros((1, states, 2, hkv, d), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(9)
    kv[:, -300:] = torch.randn((1, 300, 2, hkv, d), generator=g, device="cuda").bfloat16() * 2
    k, v = kv[:, :, 0], kv[:, :, 1]
    q = 2 * torch.randn((1, hkv, n, d), generator=g, device="cuda").bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros((1, hkv, n), device="cuda")
    svx.cross_attn(q, k, v, o, lse)
    for h in (0, 7):
        check_cross(q[:, h:h + 1], k[:, :, h:h + 1], v[:, :, h:h + 1], o[:, h:h + 1], lse[:, h:h + 1])


def shared_inputs(groups, prefix, own, hq, hkv, d, page, t, pool, seed=0):
    g = torch.Generator().manual_seed(seed)
    batch = sum(groups)
    need = [-(-n // page) for n in list(prefix) + [own] * batch]
    order = torch.randperm(sum(need) + 1, generator=g).to(torch.int32)
    far, table = (torch.full((n, max(x)), -1, dtype=torch.int32) for n, x in ((len(prefix), need[:len(prefix)]), (batch, need[len(prefix):])))
    at = 0
    for i, n in enumerate(need):
        (far[i] if i < len(prefix) else table[i - len(prefix)])[:n] = order[at:at + n]
        at += n
    if pool == "pair":  # K and V side by side
        both = torch.randn((len(order), 2, page, hkv, d), generator=g).to(t).cuda()
        k, v = both[:, 0], both[:, 1]
    elif pool == "slots":  # slots outermost
        k, v = (torch.randn((page, hkv, len(order), d), generator=g).to(t).cuda().permute(2, 0, 1, 3) for _ in range(2))
    else:
        k, v = (torch.randn((len(order), page, hkv, d), generator=g).to(t).cuda() for _ in range(2))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = 2 * torch.randn((batch, hq, 1, d), generator=g).to(t).cuda()
    return dict(q=q, k=k, v=v, far=far.cuda(), table=table.cuda(), prefix_lens=ints(list(prefix)), lens=ints([own] * batch),
                first=ints([sum(groups[:i]) for i in range(len(groups) + 1)]), o=torch.zeros_like(q),
                lse=torch.zeros((batch, hq, 1), device="cuda"))


def run_shared(c, s, **kw):
    c.decode_shared(s["q"], s["far"], s["prefix_lens"], s["first"], s["table"], s["lens"], s["o"], s["lse"], **kw)


def check_shared(s, rows=None):
    batch, hq, _, d = s["q"].shape
    group = hq // s["k"].shape[2]
    first = s["first"].tolist()
    for b in range(batch):
        mine = [slots_of(s[x], s["table"][b], int(s["lens"][b])) for x in "kv"]
        for p, n in enumerate(s["prefix_lens"].tolist()):
            if first[p] <= b < first[p + 1]:
                mine = [torch.cat((slots_of(s[x], s["far"][p], n), y)) for x, y in zip("kv", mine)]
        for h in range(s["k"].shape[2]):
            x = slice(h * group, (h + 1) * group)
            want = attend64(s["q"][b, x, 0], mine[0][:, h], mine[1][:, h], d ** -0.5)
            near(s["o"][b, x, 0], s["lse"][b, x, 0], want, p_error(rows or batch * group, s["q"].dtype), len(mine[0]))


@pytest.mark.parametrize("pool", ["token", "pair", "slots"])
@pytest.mark.parametrize("page", [1, 8, 16, 48, 64, 128, 256, 100])
def test_pages_and_pools_of_many_rows(svx, page, pool):
    """Pages that make 16, 64 or 128 slots of a tile's box, or none; pools in other orders."""
    for groups, hq, hkv, d, t in (((9, 4), 8, 2, 128, torch.float16), ((70,), 4, 1, 64, torch.bfloat16)):
        s = shared_inputs(groups, (400, 131)[:len(groups)], 19, hq, hkv, d, page, t, pool, seed=page)
        c = svx.PagedCache(s["k"], s["v"])
        run_shared(c, s)
        check_shared(s)
        assert not c.check()


def test_a_page_that_is_not_there_spoils_its_prefix_only(svx):
    s = shared_inputs((20, 21), (640, 900), 33, 4, 1, 128, 16, torch.bfloat16, "token", seed=3)
    c = svx.PagedCache(s["k"], s["v"])
    run_shared(c, s)
    check_shared(s)
    assert not c.check()
    s["far"][0, 7] = -1
    s["far"][0, 9] = s["k"].shape[0]
    run_shared(c, s)
    assert c.check()
    good = {**s, "q": s["q"][20:], "o": s["o"][20:], "lse": s["lse"][20:], "table": s["table"][20:], "lens": s["lens"][20:],
            "far": s["far"][1:], "prefix_lens": s["prefix_lens"][1:], "first": torch.tensor([0, 21])}
    check_shared(good, rows=41 * 4)  # (of the call)


def test_values_that_are_not_finite_stay_with_their_rows(svx):
    """A query that is not a number spoils its own rows alone, among 40 and among 200 others of the same product."""
    for batch in (10, 50):
        s = shared_inputs((batch,), (500,), 20, 4, 1, 64, 32, torch.bfloat16, "token", seed=4)
        s["q"][3, 1] = float("nan")
        c = svx.PagedCache(s["k"], s["v"])
        run_shared(c, s)
        assert s["o"][3, 1].isnan().all()
        s["q"][3, 1], s["o"][3, 1] = 0, 0
        clean = {**s, "o": torch.zeros_like(s["o"]), "lse": torch.zeros_like(s["lse"])}
        run_shared(c, clean)
        clean["o"][3, 1] = 0
        assert torch.equal(clean["o"], s["o"])


def test_the_checked_library_finds_rows_past_a_clipped_extent(svx):
    """svx_debug_clip_paged: states and pages described as shorter than they are.  The checked library reports it and reads nothing there."""
    def clip(n):
        assert svx.lib.svx_debug_clip_paged(2, n) == svx.OK

    for n in (2, 40):
        q, k, v = (torch.randn(s, device="cuda").bfloat16() for s in ((1, 2, n, 64), (1, 300, 1, 64), (1, 300, 1, 64)))
        o, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        try:
            clip(64 * 299)
            svx.cross_attn(q, k, v, o, status=status)
        finally:
            clip(-1)
        assert (status.item() != 0) == CHECKED
        status.zero_()
        svx.cross_attn(q, k, v, o, status=status)
        assert status.item() == 0
    for batch in (3, 40):
        s = shared_inputs((batch,), (200,), 10, 2, 1, 64, 16, torch.bfloat16, "token", seed=5)
        c = svx.PagedCache(s["k"], s["v"])
        try:
            clip(64 * 16)
            run_shared(c, s)
        finally:
            clip(-1)
        assert c.check() == CHECKED
        run_shared(c, s)
        check_shared(s)
        assert not c.check()


def test_structs_with_pointers_of_no_device_memory(svx):
    """The C calls check what the binding has not: host memory is refused."""
    s = shared_inputs((3,), (40,), 5, 4, 2, 64, 16, torch.bfloat16, "token")
    host = torch.zeros(4096, dtype=torch.float32)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    p = svx.Pages(s["k"].data_ptr(), s["v"].data_ptr(), s["table"].data_ptr(), torch.zeros(1, dtype=torch.int32, device="cuda").data_ptr(),
                  16 * 128, 128, 64, s["k"].shape[0], 16, s["table"].shape[1], 2, 64, 0, 0, 0, 0)
    f = svx.Prefixes(s["far"].data_ptr(), s["prefix_lens"].data_ptr(), s["first"].data_ptr(), 0, 1, s["far"].shape[1])
    args = lambda lse: (ctypes.byref(p), 3, 4, s["q"].data_ptr(), ctypes.byref(f), s["lens"].data_ptr(), 0, 0.0, s["o"].data_ptr(), lse,  # noqa: E731
                        ws.data_ptr(), ws.numel(), None)
    torch.cuda.synchronize()
    assert svx.lib.svx_paged_decode_shared(*args(host.data_ptr())) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_paged_decode_shared(*args(s["lse"].data_ptr())) == svx.OK
    torch.cuda.synchronize()
    check_shared(s)


# ------------------------------------------------------------------ a layer

def test_a_decoder_layer_over_branches_of_one_prompt(svx):
    """What the operators are for, together: 6 branches of one prompt, each with slots of its own, and one encoded input that all of them
    attend to; three tokens each.  Every step is checked on the inputs that it really had, and the same steps captured and replayed
    give the same."""
    B, D, hq, hkv, d, page, states, prompt = 6, 512, 8, 2, 64, 16, 333, 150
    t = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s, scale=1.0: (scale * torch.randn(s, generator=g, device="cuda")).to(t)  # noqa: E731
    w = {name: r(*shape, scale=shape[0] ** -0.5) for name, shape in dict(qkv=(D, (hq + 2 * hkv) * d), o=(hq * d, D), cq=(D, hq * d),
                                                                         ckv=(D, 2 * hkv * d), co=(hq * d, D)).items()}
    norm = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(t) for _ in range(4)]
    gate = torch.tensor([0.5], dtype=t, device="cuda")
    kv = (r(1, states, D) @ w["ckv"]).view(1, states, 2, hkv, d)
    live = torch.rand((1, states), generator=g, device="cuda") < 0.9
    pages = 2 + -(-prompt // page) + 2 * B
    kp, vp = (torch.zeros((pages, page, hkv, d), dtype=t, device="cuda") for _ in range(2))
    c = svx.PagedCache(kp, vp)
    rope = svx.Rope(d)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    far = torch.arange(-(-prompt // page), dtype=torch.int32, device="cuda")[None]
    table = ints([[far.shape[1] + 2 * b, far.shape[1] + 2 * b + 1] for b in range(B)])
    first, prefix_lens = ints([0, B]), ints([prompt])
    # the prompt into the prefix's pages
    x = r(1, prompt, D)
    heads = (x @ w["qkv"]).view(1, prompt, hq + 2 * hkv, d)
    c.append(heads[:, :, :hq], heads[:, :, hq:hq + hkv], heads[:, :, hq + hkv:], torch.arange(prompt, dtype=torch.int32, device="cuda")[None],
             rope, far, ints([0]), torch.empty((1, hq, prompt, d), dtype=t, device="cuda"))

    h = r(B, D)
    lens, pos = ints([0] * B), ints([[prompt]] * B)
    buf = {k: torch.empty((B, D), dtype=t, device="cuda") for k in ("x0", "x1", "x2", "h1", "h2", "out", "cout")}
    q1, a1 = (torch.empty((B, hq, 1, d), dtype=t, device="cuda") for _ in range(2))
    l1, a2, l2 = torch.empty((B, hq, 1), device="cuda"), torch.empty((1, B, hq, d), dtype=t, device="cuda"), torch.empty((1, hq, B), device="cuda")
    proj, cq = torch.empty((B, 1, hq + 2 * hkv, d), dtype=t, device="cuda"), torch.empty((1, B, hq, d), dtype=t, device="cuda")

    def step():
        svx.residual_norm(h, None, None, buf["x0"], norm=norm[0])
        torch.matmul(buf["x0"], w["qkv"], out=proj.view(B, -1))
        c.append(proj[:, :, :hq], proj[:, :, hq:hq + hkv], proj[:, :, hq + hkv:], pos, rope, table, lens, q1)
        lens.add_(1)
        pos.add_(1)
        c.decode_shared(q1, far, prefix_lens, first, table, lens, a1, l1)
        torch.matmul(a1.view(B, -1), w["o"], out=buf["out"])
        svx.residual_norm(h, buf["out"], buf["h1"], buf["x1"], norm=norm[1])
        torch.matmul(buf["x1"], w["cq"], out=cq.view(B, -1))
        # the branches' tokens as tokens of the one encoded input
        svx.cross_attn(cq.transpose(1, 2), kv[:, :, 0], kv[:, :, 1], a2.transpose(1, 2), l2, mask=live)
        torch.matmul(a2.view(B, -1), w["co"], out=buf["cout"])
        svx.residual_norm(buf["h1"], buf["cout"], buf["h2"], buf["x2"], norm=norm[2], post_norm=norm[3], post_eps=1e-6, gate=gate,
                          act="tanh")
        h.copy_(buf["h2"])

    start = h.clone()
    seen = []
    for n in range(1, 4):
        before = h.clone()
        step()
        s = dict(q=q1, k=kp, v=vp, far=far, table=table, prefix_lens=prefix_lens, lens=lens, first=first, o=a1, lse=l1)
        check_shared(s)
        at = live[0].nonzero()[:, 0]
        for i in range(hkv):
            heads_ = slice(i * hq // hkv, (i + 1) * hq // hkv)
            want = attend64(cq[0, :, heads_].transpose(0, 1).reshape(-1, d), kv[0, at, 0, i], kv[0, at, 1, i], d ** -0.5)
            near(a2[0, :, heads_].transpose(0, 1).reshape(-1, d), l2[0, heads_].reshape(-1), want, p_error(B * hq // hkv, t), len(at))
        u = torch.finfo(t).eps / 2
        h1 = before.double() + buf["out"].double()
        assert ((buf["h1"].double() - h1).abs() <= h1.abs() * u + (before.double().abs() + buf["out"].double().abs()) * 2.0 ** -22).all()
        y = buf["cout"].double()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * norm[3].double() * math.tanh(0.5)
        h2 = buf["h1"].double() + y
        assert ((buf["h2"].double() - h2).abs() <= h2.abs() * u + buf["h1"].double().abs() * 2.0 ** -22 + y.abs() * 2.0 ** -16).all()
        seen.append(h.clone())
    assert not c.check()
    # the same three tokens again, captured once
    h.copy_(start)
    lens.zero_()
    pos.fill_(prompt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = kp.clone()
    with torch.cuda.graph(graph):
        step()
    h.copy_(start)
    lens.zero_()
    pos.fill_(prompt)
    kp.copy_(keep)
    for want in seen:
        graph.replay()
        assert torch.equal(h, want)
    assert not c.check()


def test_prefixes_unlike_their_average(svx):
    """Items of 128 rows by the average, where one prefix has more; prefixes without requests, more of them than requests; query heads
    that fill a row tile by themselves; several row tiles whose halves are shared out over the CTAs."""
    bf16, fp16 = torch.bfloat16, torch.float16
    for groups, prefix, hq, hkv, d, page, t, rows in (((70, 1, 0, 2), (700, 300, 50, 129), 4, 1, 128, 16, bf16, 73),
                                                      ((1, 0, 0, 2, 0, 0, 0, 1), (300, 5, 6, 1000, 7, 8, 9, 128), 64, 1, 64, 32, fp16, 64),
                                                      ((2, 1), (513, 40), 130, 1, 128, 24, bf16, 195),
                                                      ((150,), (5000,), 8, 2, 64, 64, fp16, 600)):
        s = shared_inputs(groups, prefix, 21, hq, hkv, d, page, t, "token", seed=len(groups))
        c = svx.PagedCache(s["k"], s["v"])
        run_shared(c, s, max_len=21, max_prefix=max(prefix))
        check_shared(s, rows=rows)
        assert not c.check()


def test_side_by_side_with_a_round(svx):
    """Kernels that hold tensor memory on three streams at a time: a round's, those of states and those of shared prefixes."""
    hq, hkv, d, nq, hist = 8, 2, 128, 5, (900, 1300)
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    rounds = dict(q=r(2, hq, nq, d), k=[r(n, hkv, d) for n in hist], v=[r(n, hkv, d) for n in hist], kc=r(2, nq, hkv, d), vc=r(2, nq, hkv, d))
    q, k, v = r(2, 8, 200, 64), r(2, 700, 2, 64), r(2, 700, 2, 64)
    s = shared_inputs((40,), (3000,), 33, 8, 2, 128, 16, torch.bfloat16, "token", seed=9)
    c = svx.PagedCache(s["k"], s["v"])
    streams = [torch.cuda.Stream() for _ in range(3)]

    with svx.Verifier(2, hq, hkv, d, nq, 512, compute_stream=streams[0]) as verifier:
        def go(a, b, e):
            out = dict(ro=torch.empty_like(rounds["q"]), rl=torch.empty((2, hq, nq), device="cuda"), co=torch.empty_like(q),
                       cl=torch.empty((2, 8, 200), device="cuda"), so=torch.zeros_like(s["o"]), sl=torch.zeros_like(s["lse"]))
            torch.cuda.synchronize()
            for _ in range(4):
                with torch.cuda.stream(a):
                    verifier.run_round(rounds["q"], hist, rounds["k"], rounds["v"], 512, out["ro"], out["rl"], cand_k=rounds["kc"], cand_v=rounds["vc"])
                svx.cross_attn(q, k, v, out["co"], out["cl"], stream=b)
                run_shared(c, {**s, "o": out["so"], "lse": out["sl"]}, stream=e)
            torch.cuda.synchronize()
            return out

        alone = go(streams[0], streams[0], streams[0])
        for _ in range(3):
            for name, x in go(*streams).items():
                assert torch.equal(x, alone[name]), name
    check_cross(q, k, v, alone["co"], alone["cl"])
    check_shared({**s, "o": alone["so"], "lse": alone["sl"]})


def test_requests_without_states_among_many_tokens(svx):
    """Rows that have no keys are many CTAs' work: among requests that have some, alone, and without any state at all."""
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.float16)  # noqa: E731
    q, k, v = r(35, 6, 700, 64), r(35, 130, 2, 64), r(35, 130, 2, 64)
    for lens in ([0, 130, 0, 40] + [0] * 29 + [1, 0], [0] * 35):
        o = torch.full((35, 700, 6, 64), 3.0, dtype=q.dtype, device="cuda").transpose(1, 2)
        lse = torch.full((35, 6, 700), 3.0, device="cuda")
        svx.cross_attn(q, k, v, o, lse, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        check_cross(q, k, v, o, lse, seen=torch.arange(130, device="cuda") < torch.tensor(lens, device="cuda")[:, None])
    o.fill_(3)
    lse.fill_(3)
    svx.cross_attn(q, k[:, :0], v[:, :0], o, lse)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [20, 150])
@pytest.mark.parametrize("hold", [math.nan, math.inf, 6e4])
def test_what_hidden_states_hold(svx, n, d, hold):
    """Hidden states of whole tiles, of parts of tiles, behind the lengths, and all of a request's; none of them counts."""
    g = torch.Generator(device="cuda").manual_seed(n + d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.float16)  # noqa: E731
    q, k, v = r(5, 4, n, d), r(5, 700, 2, d), r(5, 700, 2, d)
    lens = torch.tensor([700, 640, 300, 700, 129], dtype=torch.int32, device="cuda")
    mask = torch.rand((5, 700), generator=g, device="cuda") < 0.7
    mask[0, :128] = False
    mask[1, 128:256] = True
    mask[3] = False
    seen = mask & (torch.arange(700, device="cuda") < lens[:, None])
    k[~seen], v[~seen] = hold, -hold
    o, lse = torch.full_like(q, 3.0), torch.full((5, 4, n), 3.0, device="cuda")
    svx.cross_attn(q, k, v, o, lse, lens=lens, mask=mask)
    check_cross(q, k, v, o, lse, seen=seen)
    assert (o[3] == 0).all() and (lse[3] == -math.inf).all()
