"""The paged-cache operators as a program uses them: a Draft's whole loop over its cache, a round fed by qk_norm_rope, CUDA graphs,
other streams and threads, far offsets, and the refusals that need tensors on a device.  Error bounds as in
test_gpu_paged.py; where one call's output feeds another, the reference takes the GPU's own tensors."""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from helpers import check_parity
from paged_reference import decode64, evict64, heads64, rows_of
from test_gpu_paged import (DECODE, check_decode, decode_inputs, evict_inputs, heads_inputs, heads_reference, make_pool, make_table,
                            near, run_decode, unit)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_draft_loop_append_decode_evict(svx):
    """Prompt in, tokens one at a time with weights accumulated, eviction when the budget is passed, on and on: after each step the
    cache, its positions and weights are what the definitions make of the GPU's own previous state."""
    g = torch.Generator().manual_seed(11)
    B, hq, hkv, d, page, budget, sink, recent = 2, 6, 2, 64, 8, 40, 2, 8
    t, room = torch.bfloat16, 64
    table, total = make_table(g, [room, room], page)
    kp, vp = make_pool(g, total, page, hkv, d, t), make_pool(g, total, page, hkv, d, t)
    cache, rope = svx.PagedCache(kp, vp), svx.Rope(d)
    inv = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(t)
    acc = torch.full((B, hkv, room), 99.0, device="cuda")
    sp = torch.full((B, hkv, room), -7, dtype=torch.int32, device="cuda")
    table_d, lens, nxt = table.cuda(), i32([0, 0]), i32([0, 0])
    held = [0, 0]

    def step(n, new):
        nonlocal held
        qkv = (2 * torch.randn((B, n, hq + 2 * hkv, d), generator=g)).to(t)
        pos = nxt.cpu()[:, None] + torch.arange(n, dtype=torch.int32)[None]
        x, q = qkv.cuda(), torch.zeros((B, hq, n, d), dtype=t, device="cuda")
        cache.append(x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], pos.cuda().contiguous(), rope, table_d, lens, q,
                     q_norm=w.cuda(), k_norm=w.cuda(), n_new=i32(new), acc=acc, slot_pos=sp)
        for b in range(B):
            m, s = new[b], held[b]
            kk, size = heads64(qkv[b, :m, hq:hq + hkv], w, 1e-6, pos[b, :m], inv, False)
            near(rows_of(kp.cpu(), table[b], s + m)[s:], kk, size, t)
            assert torch.equal(rows_of(vp.cpu(), table[b], s + m)[s:], qkv[b, :m, hq + hkv:])
            assert (acc[b, :, s:s + m] == 0).all() and torch.equal(sp[b, :, s:s + m].cpu(), pos[b, :m].expand(hkv, m))
            held[b] += m
        lens.add_(i32(new))
        nxt.add_(i32(new))
        return q

    step(37, [37, 21])
    for turn in range(6):
        q = step(1, [1, 1])
        before, k64, v64 = acc.cpu(), kp.cpu(), vp.cpu()
        o, lse = torch.zeros((B, hq, 1, d), dtype=t, device="cuda"), torch.zeros((B, hq, 1), device="cuda")
        cache.decode(q, table_d, lens, o, lse, acc_in=acc, acc_out=acc)
        want = decode64(q.cpu(), k64, v64, table, held, d ** -0.5, before)
        case = (tuple(held), hq, hkv, d, page, "bf16", "token", False)
        check_decode(case, (o, lse, None), want, None)
        err = (acc.cpu().double() - want[2]).abs()
        assert (err <= 1e-4).all()
        if turn in (2, 5):  # more tokens came in than the budget holds
            extra = step(9, [9, 3])
            assert extra.shape == (B, hq, 9, d)
        if max(held) > budget:
            a0, p0, k0, v0 = acc.cpu(), sp.cpu(), kp.cpu(), vp.cpu()
            cache.evict(table_d, lens, budget, sink, recent, nxt, acc, sp, acc, sp, lens)
            assert lens.tolist() == [min(n, budget) for n in held]
            for b in range(B):
                m = min(held[b], budget)
                for h in range(hkv):
                    order = evict64(a0[b, h].numpy(), p0[b, h].numpy(), held[b], int(nxt[b]), budget, sink, recent)
                    assert torch.equal(sp[b, h, :m].cpu(), p0[b, h][order]) and torch.equal(acc[b, h, :m].cpu(), a0[b, h][order])
                    assert torch.equal(rows_of(kp.cpu(), table[b], m)[:, h], rows_of(k0, table[b], held[b])[order, h])
                    assert torch.equal(rows_of(vp.cpu(), table[b], m)[:, h], rows_of(v0, table[b], held[b])[order, h])
                held[b] = m
    assert not cache.check()


def test_a_round_fed_by_qk_norm_rope(svx):
    """q and candidate K/V of a verification round come out of qk_norm_rope in the layout that the round takes."""
    g = torch.Generator().manual_seed(12)
    B, nq, hq, hkv, d = 2, 5, 8, 2, 128
    hist = [300, 77]
    t = torch.bfloat16
    qkv = torch.randn((B, nq, hq + 2 * hkv, d), generator=g).to(t).cuda()
    pos = torch.stack([torch.arange(n, n + nq, dtype=torch.int32) for n in hist]).cuda()
    q = torch.empty((B, hq, nq, d), dtype=t, device="cuda")
    kc, vc = (torch.empty((B, nq, hkv, d), dtype=t, device="cuda") for _ in range(2))
    svx.qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], pos, svx.Rope(d, theta=1e6), q, kc, vc)
    torch.cuda.synchronize()
    kh, vh = ([torch.randn((n, hkv, d), generator=g).to(t).cuda() for n in hist] for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty((B, hq, nq), device="cuda")
    with svx.Verifier(B, hq, hkv, d, nq, 128) as v:
        v.run_round(q, hist, kh, vh, 128, o, lse, cand_k=kc, cand_v=vc, timeout_ms=60000)
    torch.cuda.synchronize()
    f = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    o_ref, l_ref = O.verify_attention(f(q), [f(x) for x in kh], [f(x) for x in vh], f(kc), f(vc), O.visibility_table(B, nq, None),
                                      scale=d ** -0.5)
    check_parity(f(o), f(lse), o_ref, l_ref)


def test_one_token_agrees_with_a_round_over_the_same_history(svx):
    """A paged cache in order is a history: decode = a round of one query without candidates."""
    case = ((700, 129), 16, 4, 128, 16, "bf16", "token", False)
    table, kp, vp, k64, v64, q, _ = decode_inputs(case, seed=13)
    o, lse, _ = run_decode(svx, case, table, kp, vp, q, None)
    hist = [rows_of(k64, table[b], n).cuda().contiguous() for b, n in enumerate(case[0])]
    vals = [rows_of(v64, table[b], n).cuda().contiguous() for b, n in enumerate(case[0])]
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    svx.verify_static(q.cuda().contiguous(), case[0], hist, vals, o2, l2)
    torch.cuda.synchronize()
    f = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    check_parity(f(o), f(lse), f(o2), f(l2))


def test_captured_step_follows_the_lengths(svx):
    """append + decode + evict captured once; replays follow the lengths, slots and tables on the device."""
    g = torch.Generator().manual_seed(14)
    B, hq, hkv, d, page, room, budget = 3, 8, 2, 128, 16, 160, 96
    t = torch.float16
    table, total = make_table(g, [room] * B, page)
    kp, vp = make_pool(g, total, page, hkv, d, t), make_pool(g, total, page, hkv, d, t)
    cache, rope, st = svx.PagedCache(kp, vp), svx.Rope(d), torch.cuda.Stream()
    qkv, pos = torch.zeros((B, 1, hq + 2 * hkv, d), dtype=t, device="cuda"), i32([[0]] * B)
    start, lens, nxt = i32([0] * B), i32([1] * B), i32([1] * B)
    acc, sp = torch.rand((B, hkv, room), device="cuda"), torch.zeros((B, hkv, room), dtype=torch.int32, device="cuda")
    table_d = table.cuda()
    q, o, lse = (torch.zeros(s, dtype=x, device="cuda") for s, x in (((B, hq, 1, d), t), ((B, hq, 1, d), t), ((B, hq, 1), torch.float32)))
    acc2, sp2, len2 = acc.clone(), sp.clone(), lens.clone()

    def step():
        cache.append(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], pos, rope, table_d, start, q, acc=acc, slot_pos=sp)
        cache.decode(q, table_d, lens, o, lse, acc_in=acc, acc_out=acc)
        cache.evict(table_d, lens, budget, 1, 16, nxt, acc, sp, acc2, sp2, len2)

    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for lens_now in ([5, 1, 96], [97, 160, 1], [160, 100, 40]):
        x = torch.randn((B, 1, hq + 2 * hkv, d), generator=g).to(t)
        qkv.copy_(x)
        lens.copy_(torch.tensor(lens_now, dtype=torch.int32))
        start.copy_(lens - 1)
        pos.copy_(lens[:, None] + 1000)
        nxt.copy_(lens + 1001)
        acc.copy_(torch.rand((B, hkv, room), generator=g))
        sp.copy_(torch.arange(room, dtype=torch.int32).expand(B, hkv, room))
        before = acc.cpu()
        k_before, v_before = kp.cpu(), vp.cpu()
        graph.replay()
        torch.cuda.synchronize()
        # the reference on the state after append (evict moved rows of it later: redo the append from the inputs)
        k64, v64, a64, p64 = k_before.clone(), v_before.clone(), before.clone(), torch.arange(room, dtype=torch.int32).expand(B, hkv, room).clone()
        inv = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
        for b, n in enumerate(lens_now):
            kk, size = heads64(x[b, :, hq:hq + hkv], None, 1e-6, pos[b].cpu(), inv, False)
            at = (int(table[b, (n - 1) // page]), (n - 1) % page)
            order0 = [evict64(acc.cpu()[b, h].numpy(), np.where(np.arange(room) == n - 1, n + 1000, np.arange(room)), n, n + 1001, budget, 1, 16)
                      for h in range(hkv)]
            for h in range(hkv):  # where the new row went, if eviction moved it
                new_slot = order0[h].index(n - 1)
                got = kp[int(table[b, new_slot // page]), new_slot % page, h].cpu()
                near(got[None, None], kk[:, h:h + 1], size[:, h:h + 1], t)
                k64[at[0], at[1], h], v64[at[0], at[1], h] = got, x[b, 0, hq + hkv + h]
            a64[b, :, n - 1], p64[b, :, n - 1] = 0, n + 1000
            for h in range(hkv):
                m = min(n, budget)
                assert torch.equal(sp2[b, h, :m].cpu(), p64[b, h][order0[h]]) and int(len2[b]) == m
        case = (tuple(lens_now), hq, hkv, d, page, "fp16", "token", False)
        check_decode(case, (o, lse, None), decode64(q.cpu(), k64, v64, table, lens_now, d ** -0.5), None)
    assert not cache.check()


def test_streams_graphs_and_threads_at_once(svx):
    """One cache object, calls whose work overlaps: on two streams, from two threads, and in two graphs replayed side by side;
    each call has a workspace of its own."""
    cases = [((3000, 900), 8, 2, 128, 16, "bf16", "token", True), ((40, 2500), 8, 2, 128, 16, "bf16", "token", True)]
    table, kp, vp, k64, v64, q, acc = decode_inputs(((3000, 2500), 8, 2, 128, 16, "bf16", "token", True), seed=15)
    # junk behind the lengths is the tests' own; make every slot finite so that both cases may read it
    kp.nan_to_num_(0.0, 0.0, 0.0)
    vp.nan_to_num_(0.0, 0.0, 0.0)
    cache = svx.PagedCache(kp, vp)
    alone = [run_decode(svx, c, table, kp, vp, q, acc, cache=cache) for c in cases]
    qd, td, ad = q.cuda(), table.cuda(), acc.cuda()
    lens = [i32(list(c[0])) for c in cases]
    outs = [(torch.zeros_like(alone[0][0]), torch.zeros_like(alone[0][1]), torch.full_like(ad, 7.0)) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def go(i, n, explicit):
        o, lse, out = outs[i]
        for _ in range(n):
            if explicit:
                cache.decode(qd, td, lens[i], o, lse, acc_in=ad, acc_out=out, stream=streams[i])
            else:
                with torch.cuda.stream(streams[i]):
                    cache.decode(qd, td, lens[i], o, lse, acc_in=ad, acc_out=out)

    def check():
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], alone[i]))
            for x in outs[i][:2]:
                x.zero_()
            outs[i][2].fill_(7.0)

    for explicit in (False, True):
        for _ in range(20):
            go(0, 1, explicit)
            go(1, 1, explicit)
        check()
    threads = [threading.Thread(target=go, args=(i, 30, i == 0)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    check()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            go(i, 3, False)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    check()
    assert not cache.check()


def test_offsets_beyond_32_bits(svx):
    """A pool of more than 2^32 bytes a side, the request's pages at both of its ends, and a status that stays clear."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 31) // (page * hkv * d) + 300  # elements of one pool pass 2^31
    kp, vp = (torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(16)
    ids = [n_pages - 1, 0, n_pages - 2, 1, n_pages - 3]
    n = 4 * page + 7
    for i in ids:
        for pool in (kp, vp):
            pool[i] = torch.randn((page, hkv, d), generator=g).to(torch.bfloat16).cuda()
    table = torch.tensor([ids], dtype=torch.int32)
    small_k, small_v = (torch.stack([pool[i] for i in ids]).cpu() for pool in (kp, vp))
    order = torch.arange(5, dtype=torch.int32)[None]
    cache = svx.PagedCache(kp, vp)
    q = torch.randn((1, 16, 1, d), generator=g).to(torch.bfloat16)
    o, lse = torch.zeros((1, 16, 1, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 16, 1), device="cuda")
    cache.decode(q.cuda(), table.cuda(), i32([n]), o, lse)
    check_decode(((n,), 16, hkv, d, page, "bf16", "token", False), (o, lse, None),
                 decode64(q, small_k, small_v, order, [n], d ** -0.5), None)
    room = 5 * page
    acc = torch.rand((1, hkv, room), generator=g)
    pos = torch.arange(room, dtype=torch.int32).expand(1, hkv, room).contiguous()
    a, p, ln = acc.cuda(), pos.cuda(), i32([n])
    cache.evict(table.cuda(), ln, 100, 0, 0, i32([n]), a, p, a, p, ln)
    for h in range(hkv):
        want = evict64(acc[0, h].numpy(), pos[0, h].numpy(), n, n, 100, 0, 0)
        rows = rows_of(torch.stack([kp[i] for i in ids]).cpu(), order[0], 100)[:, h]
        assert torch.equal(rows, rows_of(small_k, order[0], n)[want, h]) and ln.tolist() == [100]
    x = torch.randn((1, 1, 16 + 2 * hkv, d), generator=g).to(torch.bfloat16).cuda()
    qo = torch.empty((1, 16, 1, d), dtype=torch.bfloat16, device="cuda")
    cache.append(x[:, :, :16], x[:, :, 16:24], x[:, :, 24:], i32([[5]]), svx.Rope(d), table.cuda(), i32([2 * page + 3]), qo)
    assert torch.equal(vp[n_pages - 2, 3], x[0, 0, 24:]) and not cache.check()


def test_append_out_of_room_is_reported_and_written_nowhere(svx):
    g = torch.Generator().manual_seed(17)
    page, hkv, d, t = 4, 2, 64, torch.bfloat16
    kp, vp = make_pool(g, 6, page, hkv, d, t), make_pool(g, 6, page, hkv, d, t)
    k0, v0 = kp.clone(), vp.clone()
    cache = svx.PagedCache(kp, vp)
    x = torch.randn((3, 2, 8, d), generator=g).to(t).cuda()
    qo = torch.zeros((3, 4, 2, d), dtype=t, device="cuda")
    acc = torch.ones((3, hkv, 8), device="cuda")
    args = (x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], i32([[0, 1]] * 3), svx.Rope(d))
    # past the table's room, before its start, and on a page that the pool does not have
    cache.append(*args, i32([[0, 1], [2, 3], [99, -1]]), i32([8, -2, 1]), qo, acc=acc)
    assert cache.check() and not cache.check()
    assert torch.equal(kp, k0) and torch.equal(vp, v0) and (acc == 1).all()
    assert (qo != 0).any()  # q does not depend on the slots
    cache.append(*args, i32([[0, 1], [2, 3], [4, 5]]), i32([0, 4, 3]), qo, n_new=i32([3, 2, -1]))
    assert cache.check() and torch.equal(kp[4:], k0[4:])  # counts out of bounds: clamped (all, none) and reported
    assert torch.equal(vp[0, :2], x[0, :, 6:]) and torch.equal(vp[3, :2], x[1, :, 6:])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko = torch.zeros((3, 2, 2, d), dtype=t, device="cuda")
    svx.qk_norm_rope(*args[:2], None, *args[3:], qo, ko, n_new=i32([0, 1, 2]), status=status)
    assert int(status) == 0 and (ko[0] == 0).all() and (ko[1, 1] == 0).all() and (ko[2] != 0).any()
    svx.qk_norm_rope(*args[:2], None, *args[3:], qo, ko, n_new=i32([0, 1, 5]), status=status)
    assert int(status) != 0


def test_evict_keeps_the_first_of_equal_protected_slots(svx):
    """Positions that repeat can protect more slots than the budget: the first of them stay."""
    case = ((50,), 1, 64, 8, "bf16", 10, 4, 0)
    table, kp, vp, acc, pos, nxt = evict_inputs(case, "weights")
    pos[:] = 1  # all below sink
    cache = svx.PagedCache(kp, vp)
    ao, po, lo = torch.zeros_like(acc, device="cuda"), torch.zeros_like(pos, device="cuda"), i32([0])
    cache.evict(table.cuda(), i32([50]), 10, 4, 0, nxt.cuda(), acc.cuda(), pos.cuda(), ao, po, lo)
    assert torch.equal(ao[0, 0, :10].cpu(), acc[0, 0, :10]) and lo.tolist() == [10]


def test_refusals_of_tensors_on_the_device(svx):
    kp, vp = (torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = svx.PagedCache(kp, vp)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    q, o, lse, table, lens = z(1, 4, 1, 64), z(1, 4, 1, 64), z(1, 4, 1, t=torch.float32), i32([[0, 1]]), i32([3])
    acc, pos, f32 = z(1, 2, 16, t=torch.float32), z(1, 2, 16, t=torch.int32), torch.float32
    c.decode(q, table, lens, o, lse, acc_in=acc, acc_out=acc)
    bad = [dict(q=q.half()), dict(q=z(1, 4, 64)), dict(q=z(1, 3, 1, 64)), dict(q=z(2, 4, 1, 64)), dict(q=q.cpu()),
           dict(q=z(1, 8, 1, 64)[:, ::2]), dict(o=z(1, 4, 1, 128)), dict(lse=lse.double()), dict(table=table.long()), dict(table=table[0]),
           dict(table=i32([[0, 1, 2, 3]])[:, ::2]), dict(lens=lens.long()), dict(lens=i32([1, 2])), dict(acc_in=acc),
           dict(acc_in=acc, acc_out=z(1, 2, 15, t=f32)), dict(max_len=17), dict(max_len=-1), dict(scale=-1.0),
           dict(workspace=z(64, t=torch.uint8)), dict(q=None), dict(o=None)]
    for kw in bad:
        args = dict(q=q, table=table, lens=lens, o=o, lse=lse)
        args.update(kw)
        with pytest.raises((svx.SvxError, AttributeError)):
            c.decode(**args)
    n, p = svx.ctypes.c_int64(0), svx.Pages.from_buffer_copy(c._pages)
    p.table, p.max_pages = table.data_ptr(), 2
    assert svx.lib.svx_paged_decode_workspace(svx.ctypes.byref(p), 1, 4, 0, 0, svx.ctypes.byref(n)) == svx.OK
    ws = z(n.value + 256, t=torch.uint8)
    c.decode(q, table, lens, o, lse, workspace=ws)
    with pytest.raises(svx.SvxError):  # a workspace off its alignment
        c.decode(q, table, lens, o, lse, workspace=ws[8:])
    with pytest.raises(svx.SvxError):  # pages off the 16-byte grid
        flat = z(4 * 8 * 2 * 64 + 8)
        svx.PagedCache(flat[1:-7].view(4, 8, 2, 64), flat[1:-7].view(4, 8, 2, 64)).decode(q, table, lens, o, lse)
    with pytest.raises(svx.SvxError):
        svx.PagedCache(kp, vp.half())
    with pytest.raises(svx.SvxError):
        svx.PagedCache(kp.float(), vp.float())
    with pytest.raises(svx.SvxError):
        svx.PagedCache(kp[..., ::2], vp[..., ::2])
    ln, nx = i32([16]), i32([20])
    c.evict(table, ln, 8, 1, 2, nx, acc, pos, acc, pos, ln)
    for kw in (dict(budget=0), dict(sink=7, recent=2), dict(acc_in=acc.double()), dict(pos_in=pos.long()), dict(next_pos=None),
               dict(len_out=i32([1, 2])), dict(max_len=99), dict(acc_in=None), dict(pos_out=z(1, 2, 17, t=torch.int32))):
        args = dict(table=table, lens=ln, budget=8, sink=1, recent=2, next_pos=nx, acc_in=acc, pos_in=pos, acc_out=acc, pos_out=pos,
                    len_out=ln)
        args.update(kw)
        with pytest.raises(svx.SvxError):
            c.evict(**args)
    x, qo, ko, rope = z(2, 3, 8, 64), z(2, 4, 3, 64), z(2, 3, 2, 64), svx.Rope(64)
    p2 = z(2, 3, t=torch.int32)
    heads = dict(q=x[:, :, :4], k=x[:, :, 4:6], v=x[:, :, 6:], pos=p2, rope=rope, q_out=qo, k_out=ko, v_out=torch.zeros_like(ko))
    svx.qk_norm_rope(**heads)
    for kw in (dict(q=x[:, :, ::2]), dict(q=x[:, ::2, :4]), dict(k=x[:1, :, 4:6]), dict(k=x.half()[:, :, 4:6]), dict(v=x[:, :, 7:]), dict(v=None),
               dict(v_out=None), dict(pos=p2.long()), dict(pos=None), dict(q_out=qo.transpose(1, 2)), dict(q_norm=z(32)), dict(eps=None, q_norm=z(64)),
               dict(eps=-1.0), dict(n_new=z(3, t=torch.int32)), dict(rope=svx.Rope(128)), dict(k_out=None), dict(status=z(2, t=torch.int32)),
               dict(q=x[:, :, 1:5, 4:].reshape(2, 3, 4, 60))):
        with pytest.raises(svx.SvxError):
            svx.qk_norm_rope(**dict(heads, **kw))
    full = z(2, 3, 4 + 2 + 2, 64)
    with pytest.raises(svx.SvxError):  # the output inside the projection that it is read from
        svx.qk_norm_rope(full[:, :, :4], full[:, :, 4:6], full[:, :, 6:], p2, rope, full.view(-1)[:2 * 4 * 3 * 64].view(2, 4, 3, 64), ko, ko.clone())
    # tokens that are not evenly spaced over the requests
    with pytest.raises(svx.SvxError):
        y = z(2, 5, 8, 64)[:, :3]
        svx.qk_norm_rope(y[:, :, :4], y[:, :, 4:6], None, p2, rope, qo, ko)
    # C ABI: a host address where device memory is wanted is refused, unless the caller vouches for it
    host = np.zeros(64, dtype=np.int32)
    p.flags = 0
    st = svx.lib.svx_paged_decode(svx.ctypes.byref(p), 1, 4, q.data_ptr(), host.ctypes.data, 0, 0.0, o.data_ptr(), lse.data_ptr(), None,
                                  None, ws.data_ptr(), ws.numel(), None)
    assert st == svx.ERR_INVALID_ARG
    assert svx.lib.svx_paged_decode(svx.ctypes.byref(p), 1, 4, q.data_ptr(), lens.data_ptr(), 0, 0.0, o.data_ptr(), lse.data_ptr(), None,
                                    None, ws.data_ptr(), ws.numel(), None) == svx.OK
    for bad in ((1, 2), (None,) * 11, (c._pages,) * 11):  # the native calls themselves: counts and kinds of arguments
        with pytest.raises((TypeError, svx.SvxError)):
            c._native.decode(*bad)
    assert not c.check()


@pytest.mark.parametrize("case", DECODE[3:5], ids=str)
def test_explicit_workspace_and_no_set_up(svx, case):
    """A workspace full of anything does: NaN bits, then a previous call's leavings."""
    table, kp, vp, k64, v64, q, acc = decode_inputs(case, seed=18)
    want = run_decode(svx, case, table, kp, vp, q, acc)
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = run_decode(svx, case, table, kp, vp, q, acc, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_heads_rows_do_not_depend_on_the_batch(svx):
    """The same token in a batch of one and inside a large one (several heads to a warp): the same bits."""
    case = (1, 1200, 16, 4, 128, 128, False, True, "bf16", 1.0)
    qkv, pos, wq, wk, inv = heads_inputs(case, seed=19)
    rope = svx.Rope(128, inv_freq=inv)

    def go(x, p):
        b, n = p.shape
        qo, ko = torch.empty((b, 16, n, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((b, n, 4, 128), dtype=torch.bfloat16, device="cuda")
        svx.qk_norm_rope(x[:, :, :16], x[:, :, 16:20], None, p, rope, qo, ko, q_norm=wq.cuda(), k_norm=wk.cuda())
        return qo.transpose(1, 2), ko
    big = go(qkv.cuda(), pos.cuda())
    for i in (0, 1, 599, 1199):
        one = go(qkv[:, i:i + 1].cuda().contiguous(), pos[:, i:i + 1].cuda().contiguous())
        assert torch.equal(one[0], big[0][:, i:i + 1]) and torch.equal(one[1], big[1][:, i:i + 1])
    q, qs, k, ks, _ = heads_reference(case, qkv, pos, wq, wk, inv)
    near(big[0], q, qs, torch.bfloat16)
    assert unit(torch.bfloat16) == 2.0 ** -8


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_evict_in_other_layouts(svx, layout):
    """Heads outside the slots, and K and V side by side in one tensor: rows move, nothing between them does."""
    g = torch.Generator().manual_seed(20)
    page, hkv, d, n, budget = 24, 3, 64, 500, 200
    table, total = make_table(g, [n, n], page)
    kp, vp = make_pool(g, total, page, hkv, d, torch.float16, layout) if layout == "pair" else \
        tuple(make_pool(g, total, page, hkv, d, torch.float16, layout) for _ in range(2))
    k0, v0 = kp.cpu().clone(), vp.cpu().clone()
    room = table.shape[1] * page
    acc = torch.rand((2, hkv, room), generator=g)
    pos = torch.arange(room, dtype=torch.int32).expand(2, hkv, room).contiguous()
    cache = svx.PagedCache(kp, vp)
    a, p, lo = acc.cuda(), pos.cuda(), i32([0, 0])
    cache.evict(table.cuda(), i32([n, n]), budget, 3, 20, i32([n, n]), a, p, a, p, lo)
    assert not cache.check() and lo.tolist() == [budget, budget]
    for b in range(2):
        for h in range(hkv):
            order = evict64(acc[b, h].numpy(), pos[b, h].numpy(), n, n, budget, 3, 20)
            assert torch.equal(p[b, h, :budget].cpu(), pos[b, h][order])
            for t, f in enumerate(order):
                if t != f:
                    k0[int(table[b, t // page]), t % page, h] = k0[int(table[b, f // page]), f % page, h]
                    v0[int(table[b, t // page]), t % page, h] = v0[int(table[b, f // page]), f % page, h]
    assert torch.equal(kp.cpu(), k0) and torch.equal(vp.cpu(), v0)


def test_a_cache_keeps_the_memory_that_it_was_given(svx):
    """The caller's tensors get other memory: the cache still works on the first, which it holds."""
    import copy
    kp = torch.randn((4, 16, 1, 64), device="cuda", dtype=torch.bfloat16)
    vp = torch.randn_like(kp)
    q = torch.randn((1, 1, 1, 64), device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    cache = svx.PagedCache(kp, vp)
    at = kp.data_ptr()

    def step():
        o, lse = torch.empty_like(q), torch.empty((1, 1, 1), device="cuda")
        cache.decode(q, table, lens, o, lse)
        assert not cache.check()
        return o, lse
    first = step()
    kp.data, vp.data = torch.zeros_like(kp), torch.zeros_like(vp)
    del kp, vp
    junk = [torch.full((4, 16, 1, 64), 9.0, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    assert cache.k_pages.data_ptr() == at and all(j.data_ptr() != at for j in junk)
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    for name in ("k_pages", "v_pages", "status"):
        with pytest.raises(AttributeError):
            setattr(cache, name, junk[0])
    with pytest.raises(TypeError):
        copy.deepcopy(cache)
