"""The paged-cache entry points without a GPU: the rotation's fixed-point phases, the arithmetic that the kernels share
with the host, and every refusal that comes before the first CUDA call (fake addresses, which no call may follow)."""
import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest


@pytest.fixture(scope="module")
def svx():
    from speculative_decoding_verification_chunked_gb300 import build
    if not all(os.path.exists(x) for x in (build.LIB, build.LIB_CHECKED, build.LIB_TORCH)):
        build.build()
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def test_turns_are_the_fraction_of_a_turn_per_position(svx):
    """turns = inv_freq / 2 pi mod 1 in units of 2^-64, to the double's precision: pos * turns mod 2^64 then is the phase of any
    32-bit position within pos * 2^-53 turns."""
    from math import pi
    inv = [1.0, 0.5, 1e-3, 3e-7, 2 * pi, 10.0, -0.25, 0.0]
    r = svx.Rope(16, inv_freq=inv)
    for i, f in enumerate(inv):
        exact = Fraction(f) / Fraction(2 * pi)  # (2 pi itself is a double here: 2^-53 relative)
        got = Fraction(r.table.turns[i], 1 << 64)
        off = (got - exact) % 1
        off = min(off, 1 - off)
        assert off <= abs(exact) * Fraction(1, 1 << 51) + Fraction(1, 1 << 52), (f, float(off))
    assert all(r.table.turns[i] == 0 for i in range(8, 64))
    assert (r.table.rot_dim, r.table.neighbours, r.table.scale) == (16, 0, 1.0)


def test_copies_of_a_rope_have_their_own_table(svx):
    """A model that holds one may be copied and the original freed."""
    import copy
    import pickle
    r = svx.Rope(16, theta=500.0)
    for c in (copy.deepcopy(r), pickle.loads(pickle.dumps(r)), copy.copy(r)):
        assert c.address == ctypes.addressof(c.table) and list(c.table.turns) == list(r.table.turns)
    assert copy.deepcopy(r).address != r.address


def test_rope_refusals(svx):
    ok = [0.5] * 64
    for rot, inv in ((8, ok[:4]), (-16, []), (24, ok[:12]), (144, [0.5] * 72), (16, ok[:7]), (16, [float("nan")] * 8),
                     (16, [float("inf")] * 8), (16, [2.0 ** 20] * 8)):
        with pytest.raises(svx.SvxError):
            svx.Rope(rot, inv_freq=inv)
    with pytest.raises(svx.SvxError):
        svx.Rope(16, scale=float("inf"))
    assert svx.lib.svx_rope_init(None, 16, 0, (ctypes.c_double * 8)(), 1.0) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_rope_init(ctypes.byref(svx.RopeTable()), 16, 0, None, 1.0) == svx.ERR_INVALID_ARG
    assert svx.Rope(0).table.rot_dim == 0


# Addresses that no refused call may read; 256-byte aligned.
K, V, TABLE, STATUS, Q, O, LSE, LEN, ACC, ACC2, WS, POS, NEXT, POS2, LEN2, KOUT, VOUT = (0x100000000 * (i + 1) for i in range(17))


def pages(svx, **kw):
    f = dict(k=K, v=V, table=TABLE, status=STATUS, page_stride=16 * 2 * 128, tok_stride=2 * 128, head_stride=128, n_pages=10,
             page_size=16, max_pages=4, n_kv_heads=2, head_dim=128, dtype=0, device=0, flags=0, pad=0)
    f.update(kw)
    return svx.Pages(*[f[n] for n, _ in svx.Pages._fields_])


def heads(svx, **kw):
    f = dict(q=Q, k=K, v=V, q_stride=1024, k_stride=1024, v_stride=1024, q_norm=None, k_norm=None, pos=POS, n_new=None, status=None,
             n_req=2, n_tok=3, n_q_heads=4, n_kv_heads=2, head_dim=128, dtype=0, device=0, eps=1e-6, flags=0, pad=0)
    f.update(kw)
    return svx.Heads(*[f[n] for n, _ in svx.Heads._fields_])


BAD_PAGES = [dict(k=None), dict(v=None), dict(table=None), dict(status=None), dict(k=K + 8), dict(v=V + 2), dict(page_size=0),
             dict(max_pages=0), dict(page_size=1 << 16, max_pages=1 << 15), dict(n_pages=0), dict(n_pages=1 << 31),
             dict(n_kv_heads=0), dict(head_dim=96), dict(dtype=2), dict(dtype=-1), dict(tok_stride=252), dict(tok_stride=64),
             dict(head_stride=0), dict(page_stride=-4096), dict(page_stride=1 << 50), dict(page_stride=4100), dict(status=STATUS + 2)]


@pytest.mark.parametrize("bad", BAD_PAGES, ids=str)
def test_bad_pages_are_refused_by_every_call(svx, bad):
    p = ctypes.byref(pages(svx, **bad))
    refused = (svx.ERR_INVALID_ARG, svx.ERR_UNSUPPORTED)
    n = ctypes.c_int64(7)
    assert svx.lib.svx_paged_evict_workspace(p, 2, 0, 8, ctypes.byref(n)) in refused and n.value == 0
    assert svx.lib.svx_paged_decode_workspace(p, 2, 4, 0, 0, ctypes.byref(n)) in refused
    assert svx.lib.svx_paged_decode(p, 2, 4, Q, LEN, 0, 0.0, O, LSE, None, None, WS, 1 << 40, None) in refused
    assert svx.lib.svx_paged_evict(p, 2, LEN, 0, 8, 0, 0, NEXT, ACC, POS, ACC2, POS2, LEN2, WS, 1 << 40, None) in refused
    h = heads(svx, k=KOUT, v=VOUT)
    if "head_dim" not in bad and "dtype" not in bad:
        assert svx.lib.svx_paged_append(ctypes.byref(h), ctypes.byref(svx.Rope(128).table), p, LEN, O, None, None, None) in refused
    assert svx.lib.svx_last_error(None)


def test_decode_refusals(svx):
    p = ctypes.byref(pages(svx))

    def call(n_req=2, hq=4, q=Q, ln=LEN, max_len=0, scale=0.0, o=O, lse=LSE, a=None, b=None, ws=WS, size=1 << 40):
        return svx.lib.svx_paged_decode(p, n_req, hq, q, ln, max_len, scale, o, lse, a, b, ws, size, None)
    for kw in (dict(n_req=0), dict(n_req=257), dict(q=None), dict(ln=None), dict(o=None), dict(lse=None), dict(q=Q + 8),
               dict(o=O + 4), dict(lse=LSE + 2), dict(a=ACC), dict(b=ACC), dict(a=ACC, b=ACC + 64), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) in (svx.ERR_INVALID_ARG, svx.ERR_UNSUPPORTED), kw
    for kw in (dict(hq=3), dict(hq=0), dict(hq=8192), dict(max_len=-1), dict(max_len=65)):
        assert call(**kw) == svx.ERR_INVALID_ARG, kw
    n = ctypes.c_int64(0)
    assert svx.lib.svx_paged_decode_workspace(p, 2, 4, 0, 0, None) == svx.ERR_INVALID_ARG
    # too many chunks for the 32-bit plan: 256 requests x 4096 KV heads x 2^15 slots
    big = pages(svx, n_kv_heads=4096, page_stride=1 << 23, tok_stride=4096 * 128, max_pages=1 << 11)
    assert svx.lib.svx_paged_decode_workspace(ctypes.byref(big), 256, 4096, 0, 0, ctypes.byref(n)) in \
        (svx.ERR_UNSUPPORTED, svx.ERR_CUDA)


def test_evict_refusals_and_workspace(svx):
    p = ctypes.byref(pages(svx))

    def call(n_req=2, ln=LEN, max_len=0, budget=8, sink=1, recent=2, nxt=NEXT, a=ACC, q=POS, a2=ACC2, q2=POS2, l2=LEN2, ws=WS,
             size=1 << 40):
        return svx.lib.svx_paged_evict(p, n_req, ln, max_len, budget, sink, recent, nxt, a, q, a2, q2, l2, ws, size, None)
    for kw in (dict(n_req=0), dict(ln=None), dict(nxt=None), dict(a=None), dict(q=None), dict(a2=None), dict(q2=None), dict(l2=None),
               dict(budget=0), dict(budget=-3), dict(sink=-1), dict(recent=-1), dict(sink=7, recent=2), dict(max_len=65),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1), dict(max_len=-1), dict(ws=None), dict(ws=WS + 16), dict(size=16),
               dict(a2=ACC + 4), dict(q2=POS - 8), dict(l2=LEN + 4), dict(l2=NEXT), dict(l2=NEXT + 4)):
        assert call(**kw) == svx.ERR_INVALID_ARG, kw
    n = ctypes.c_int64(0)
    for max_len, budget in ((0, 8), (64, 64), (10, 64), (64, 1)):
        assert svx.lib.svx_paged_evict_workspace(p, 2, max_len, budget, ctypes.byref(n)) == svx.OK
        most = max(0, min(budget, (max_len or 64) - budget))
        assert n.value >= 2 * 2 * 4 + 2 * 4 + 2 * (2 * 2 * most * 4)
    wide = ctypes.byref(pages(svx, max_pages=1 << 16))
    assert svx.lib.svx_paged_evict_workspace(wide, 2, svx.EVICT_MAX_LEN + 1, 8, ctypes.byref(n)) == svx.ERR_UNSUPPORTED
    assert svx.lib.svx_paged_evict_workspace(wide, 2, 0, 8, ctypes.byref(n)) == svx.OK  # 0: the longest


def test_heads_refusals(svx):
    rope = svx.Rope(128)

    def dense(q_out=O, k_out=KOUT, v_out=VOUT, r=ctypes.byref(rope.table), **kw):
        return svx.lib.svx_qk_norm_rope(ctypes.byref(heads(svx, **kw)), r, q_out, k_out, v_out, None)
    bad = [dict(n_req=0), dict(n_req=257), dict(n_tok=0), dict(head_dim=80), dict(dtype=7), dict(n_kv_heads=0), dict(n_kv_heads=3),
           dict(n_q_heads=8192, n_kv_heads=1, q_stride=1 << 20), dict(q_stride=504), dict(k_stride=128), dict(v_stride=1028), dict(q_stride=1 << 60),
           dict(q=None), dict(k=None), dict(q=Q + 8), dict(v=V + 4), dict(q_out=None), dict(k_out=None), dict(k_out=KOUT + 8),
           dict(v_out=None), dict(v=None), dict(pos=None), dict(eps=float("nan")), dict(eps=-1.0, q_norm=LSE),
           dict(q_norm=LSE + 8), dict(k_norm=LSE + 2), dict(r=None),
           dict(r=ctypes.byref(rope.table), head_dim=64),                                  # rotation wider than the head
           dict(q_out=Q), dict(k_out=Q + 1024), dict(v_out=V), dict(q_out=KOUT), dict(v_out=KOUT + 512)]  # overlaps
    for kw in bad:
        assert dense(**kw) in (svx.ERR_INVALID_ARG, svx.ERR_UNSUPPORTED), kw
    p = pages(svx, k=KOUT, v=VOUT)

    def append(start=LEN, q_out=O, cache=p, **kw):
        return svx.lib.svx_paged_append(ctypes.byref(heads(svx, **kw)), ctypes.byref(rope.table), ctypes.byref(cache), start, q_out, None, None, None)
    for kw in (dict(start=None), dict(v=None), dict(n_kv_heads=1), dict(dtype=1), dict(device=1), dict(q_out=KOUT),
               dict(k=KOUT + 1024), dict(cache=pages(svx, k=KOUT, v=VOUT, head_dim=64))):
        assert append(**kw) == svx.ERR_INVALID_ARG, kw
    assert svx.lib.svx_paged_append(ctypes.byref(heads(svx)), ctypes.byref(rope.table), None, LEN, O, None, None, None) == svx.ERR_INVALID_ARG


def test_outputs_over_inputs_or_each_other_are_refused(svx):
    """Every such pair of every call, by one element at either end; the pairs that may be one buffer get past it."""
    rope = ctypes.byref(svx.Rope(128).table)
    p = ctypes.byref(pages(svx))
    row, meta, ints = 2 * 4 * 128 * 2, 2 * 2 * 64 * 4, 2 * 4

    def message():
        return svx.lib.svx_last_error(None).decode()

    def decode(q=Q, ln=LEN, o=O, lse=LSE, a=ACC, b=ACC2):
        st = svx.lib.svx_paged_decode(p, 2, 4, q, ln, 0, 0.0, o, lse, a, b, WS, 1 << 40, None)
        return st == svx.ERR_INVALID_ARG and "overlap" in message()
    assert not decode() and not decode(b=ACC)
    for kw in (dict(o=Q), dict(o=Q + row - 16), dict(o=Q - row + 16), dict(lse=Q + row - 4), dict(lse=O), dict(lse=LEN), dict(b=TABLE),
               dict(b=O - meta + 4), dict(b=ACC - meta + 4), dict(a=O), dict(lse=STATUS), dict(ln=LSE + 28), dict(ln=STATUS)):
        assert decode(**kw), kw
    for kw in (dict(o=Q + row), dict(o=Q - row), dict(lse=Q + row), dict(ln=LSE + 32), dict(b=ACC + meta)):
        assert not decode(**kw), kw

    def evict(ln=LEN, nxt=NEXT, a=ACC, q=POS, a2=ACC2, q2=POS2, l2=LEN2, ws=WS):
        st = svx.lib.svx_paged_evict(p, 2, ln, 0, 8, 1, 2, nxt, a, q, a2, q2, l2, ws, 1 << 40, None)
        return st == svx.ERR_INVALID_ARG and "overlap" in message()
    assert not evict() and not evict(a2=ACC, q2=POS, l2=LEN)
    for kw in (dict(a2=POS), dict(q2=ACC + meta - 4), dict(a2=ACC + 4), dict(q2=POS - 8), dict(l2=LEN + 4), dict(l2=NEXT), dict(l2=NEXT - 4),
               dict(a2=TABLE), dict(a2=POS2), dict(l2=ACC2 + meta - 4), dict(ws=ACC), dict(ws=LEN), dict(ws=POS2), dict(l2=STATUS), dict(q=ACC2)):
        assert evict(**kw), kw
    assert not evict(a2=ACC + meta) and not evict(l2=LEN + ints)

    def append(acc=ACC, pos=POS2, start=LEN, q_out=O, **kw):
        c = pages(svx, k=KOUT, v=VOUT)
        st = svx.lib.svx_paged_append(ctypes.byref(heads(svx, **kw)), rope, ctypes.byref(c), start, q_out, acc, pos, None)
        return st == svx.ERR_INVALID_ARG and "overlap" in message()
    assert not append()
    for kw in (dict(acc=POS), dict(pos=POS), dict(pos=ACC + 4), dict(acc=LEN - meta + 4), dict(pos=TABLE), dict(acc=O), dict(acc=STATUS),
               dict(q_out=LEN), dict(acc=Q), dict(pos=KOUT), dict(q_out=POS), dict(q_norm=O), dict(n_new=ACC)):
        assert append(**kw), kw

    def dense(q_out=O, k_out=KOUT, v_out=VOUT, **kw):
        st = svx.lib.svx_qk_norm_rope(ctypes.byref(heads(svx, **kw)), rope, q_out, k_out, v_out, None)
        return st == svx.ERR_INVALID_ARG and "overlap" in message()
    assert not dense()
    for kw in (dict(q_out=POS), dict(k_out=KOUT, q_norm=KOUT), dict(v_out=O), dict(n_new=VOUT), dict(status=O), dict(k_out=V)):
        assert dense(**kw), kw


def test_binding_refuses_tensors_off_the_gpu(svx):
    import torch
    k = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(svx.SvxError):
        svx.PagedCache(k, k)
    with pytest.raises(svx.SvxError):
        svx.PagedCache(k, k[:1])
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(svx.SvxError):
        svx.qk_norm_rope(q, q, None, torch.zeros((1, 1), dtype=torch.int32), svx.Rope(64), q, q)
    with pytest.raises(svx.SvxError):
        svx.qk_norm_rope(q.float(), q, None, torch.zeros((1, 1), dtype=torch.int32), svx.Rope(64), q, q)


def test_page_division_by_multiplication():
    """The kernels find a slot's page as (t + mulhi(t, mul)) >> l with 2^l >= page_size, mul = floor(2^32 (2^l - p) / p) + 1: the
    quotient for every t < 2^31 and page size, without overflow of the 32-bit sum."""
    rng = np.random.default_rng(0)
    for d in list(range(1, 200)) + [1000, 4097, 65535, 99991, (1 << 20) + 7, (1 << 30) - 1, 1 << 30, (1 << 31) - 1]:
        l = 0
        while (1 << l) < d:
            l += 1
        mul = ((1 << 32) * ((1 << l) - d)) // d + 1
        assert mul < 1 << 32
        t = np.concatenate([rng.integers(0, 2 ** 31, 4000), np.arange(500), np.arange(2 ** 31 - 500, 2 ** 31),
                            (np.arange(1, 500) * d) % 2 ** 31, (np.arange(1, 500) * d - 1) % 2 ** 31]).astype(np.uint64)
        total = t + ((t * np.uint64(mul)) >> np.uint64(32))
        assert total.max() < 1 << 32 and ((total >> np.uint64(l)) == t // np.uint64(d)).all(), d


def test_split_of_chunks_over_ctas():
    """begin(c) = c q + c r / used over T = q used + r tiles [0, T) exactly, and the float estimate of the CTA that holds a
    chunk is at most two steps off."""
    rng = np.random.default_rng(1)
    for _ in range(3000):
        T = int(rng.integers(1, 5000 if rng.random() < 0.7 else 2 ** 31 - 1))
        used = min(-(-T // 16), int(rng.integers(1, 257)))
        q, r = divmod(T, used)
        begin = lambda c: c * q + c * r // used  # noqa: E731
        assert begin(0) == 0 and begin(used) == T and all(begin(c) < begin(c + 1) for c in {0, used // 2, used - 1})
        for x in {0, T - 1, int(rng.integers(0, T))}:
            c, steps = min(int(np.float32(x) * (np.float32(used) / np.float32(T))), used - 1), 0
            while c + 1 < used and begin(c + 1) <= x:
                c, steps = c + 1, steps + 1
            while c > 0 and begin(c) > x:
                c, steps = c - 1, steps + 1
            assert begin(c) <= x < begin(c + 1) and steps <= 2


def histogram_cut(keys, n):
    """select_kernel's search, step by step: keep keys > cut, and of those equal to it the first `need`."""
    keys = np.asarray(keys, dtype=np.uint64)
    free = keys[keys != 0xffffffff]
    need = n - (len(keys) - len(free))
    if need <= 0:
        return 0xffffffff, n
    lo, hi = int(free.min()), int(free.max())
    span, passes = hi - lo, 0
    while True:
        shift = max(span.bit_length() - 8, 0)
        d = (keys - np.uint64(lo)) % np.uint64(1 << 32)
        bins = np.bincount((d[d <= span] >> np.uint64(shift)).astype(np.int64), minlength=256)
        assert len(bins) == 256 and passes < 4
        above = 0
        for b in range(255, -1, -1):
            if above < need <= above + bins[b]:
                break
            above += bins[b]
        need, lo, passes = need - above, lo + (b << shift), passes + 1
        if bins[b] == need:
            return lo - 1, 0
        if shift == 0:
            return lo, need
        span = min((1 << shift) - 1, hi - lo)


def test_histogram_search_finds_the_nth_largest_key():
    rng = np.random.default_rng(2)
    for trial in range(400):
        size = int(rng.integers(2, 400))
        kind = trial % 5
        if kind == 0:
            keys = rng.integers(1, 0xff800001, size)
        elif kind == 1:
            keys = 0x80000000 + rng.integers(0, 5, size)
        elif kind == 2:
            keys = rng.choice([0x007fffff, 0x80000000, 0xff800000, 0xfffffff0 - 0x800000], size)
        elif kind == 3:
            keys = np.full(size, int(rng.integers(1, 0xff800001)))
        else:  # the widest range, with its ends
            keys = np.concatenate([[0x007fffff, 0xff800000], rng.integers(0xff7ffff0, 0xff800001, size)])
        keys = keys.astype(np.uint64)
        if trial % 3:
            keys[rng.random(len(keys)) < 0.3] = 0xffffffff
            keys[0] = 5000  # some key is not protected
        n = int(rng.integers(1, len(keys)))
        cut, need = histogram_cut(keys, n)
        ties = np.flatnonzero(keys == cut)[:need]
        kept = sorted(np.flatnonzero(keys > cut).tolist() + ties.tolist())
        assert kept == sorted(sorted(range(len(keys)), key=lambda t: (-int(keys[t]), t))[:n])
