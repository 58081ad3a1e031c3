"""Edges of the paged-cache entry points without a GPU: exact phases, and refusals that come before the first CUDA call (fake addresses,
which no call may follow)."""
import ctypes
import os
import random
from fractions import Fraction

import pytest

# 2 pi to 60 digits, far beyond what the products below need
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(scope="module")
def svx():
    from speculative_decoding_verification_chunked_gb300 import build
    if not all(os.path.exists(x) for x in (build.LIB, build.LIB_CHECKED)):
        build.build()
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def test_turns_are_exact_for_every_frequency(svx):
    """turns is the fraction of a turn to one unit of 2^-64, so that no 32-bit position's phase is off by more than 2^-33 turns,
    for the fastest pairs that are taken too."""
    inv = [1.0, 0.1, 1e-3, 3e-7, 1e-17, 5e-324, 2.0 ** -60, 6.283185307179586, 10.0, 1e5, 524287.3, 2.0 ** 20 - 2.0 ** -32, 1048575.9999999999, 0.0,
           99999.99, 123456.789]
    for sign in (1.0, -1.0):
        r = svx.Rope(32, inv_freq=[sign * f for f in inv])
        for i, f in enumerate(inv):
            got, exact = Fraction(r.table.turns[i], 1 << 64), Fraction(sign * f) / TWO_PI
            off = (got - exact) % 1
            off = min(off, 1 - off)
            assert off <= Fraction(1, 1 << 64), (sign * f, float(off * 2 ** 64))
            for pos in (2 ** 31 - 1, -2 ** 31, 131071):
                phase = Fraction((pos * r.table.turns[i]) % (1 << 64), 1 << 64) - pos * exact
                assert min(phase % 1, 1 - phase % 1) <= Fraction(1, 1 << 33)


# ------------------------------------------------------------------ buffers that meet the pools

# Addresses that no refused call may read; 256-byte aligned.
K, V, TABLE, STATUS, Q, O, LSE, LEN, ACC, ACC2, WS, POS, NEXT, POS2, LEN2, KIN, VIN, NORM = (0x100000000 * (i + 1) for i in range(18))
POOL = 2 * (9 * 4096 + 15 * 256 + 128 + 128)  # bytes from the first row of pages() to behind its last


def pages(svx, **kw):
    f = dict(k=K, v=V, table=TABLE, status=STATUS, page_stride=16 * 2 * 128, tok_stride=2 * 128, head_stride=128, n_pages=10,
             page_size=16, max_pages=4, n_kv_heads=2, head_dim=128, dtype=0, device=0, flags=0, pad=0)
    f.update(kw)
    return svx.Pages(*[f[n] for n, _ in svx.Pages._fields_])


def heads(svx, **kw):
    f = dict(q=Q, k=KIN, v=VIN, q_stride=1024, k_stride=1024, v_stride=1024, q_norm=None, k_norm=None, pos=POS, n_new=None, status=None,
             n_req=2, n_tok=3, n_q_heads=4, n_kv_heads=2, head_dim=128, dtype=0, device=0, eps=1e-6, flags=0, pad=0)
    f.update(kw)
    return svx.Heads(*[f[n] for n, _ in svx.Heads._fields_])


def refused(svx, status, words=("overlap", "share memory")):
    return status == svx.ERR_INVALID_ARG and any(w in svx.lib.svx_last_error(None).decode() for w in words)


def decode(svx, cache=None, q=Q, ln=LEN, o=O, lse=LSE, a=ACC, b=ACC2, ws=WS, scale=0.0):
    c = cache or pages(svx)
    return svx.lib.svx_paged_decode(ctypes.byref(c), 2, 4, q, ln, 0, scale, o, lse, a, b, ws, 1 << 30, None)


@pytest.mark.parametrize("pool", [K, V], ids=["k", "v"])
def test_decode_refuses_outputs_in_the_pools(svx, pool):
    row, meta = 2 * 4 * 128 * 2, 2 * 2 * 64 * 4
    for kw in (dict(o=pool), dict(o=pool + POOL - 16), dict(o=pool - row + 16), dict(lse=pool), dict(lse=pool + POOL - 4), dict(b=pool),
               dict(a=pool, b=pool), dict(b=pool - meta + 4),
               dict(cache=pages(svx, status=pool + 64))):
        assert refused(svx, decode(svx, **kw)), kw
    for kw in (dict(o=pool + POOL), dict(o=pool - row), dict(lse=pool + POOL), dict(b=pool + POOL), dict(q=pool),
               dict(cache=pages(svx, k=V))):  # (one buffer read twice is no overlap)
        assert not refused(svx, decode(svx, **kw)), kw


def evict(svx, cache=None, ln=LEN, nxt=NEXT, a=ACC, q=POS, a2=ACC2, q2=POS2, l2=LEN2, ws=WS):
    c = cache or pages(svx)
    return svx.lib.svx_paged_evict(ctypes.byref(c), 2, ln, 0, 8, 1, 2, nxt, a, q, a2, q2, l2, ws, 1 << 30, None)


@pytest.mark.parametrize("pool", [K, V], ids=["k", "v"])
def test_evict_refuses_buffers_in_the_pools(svx, pool):
    """Eviction writes the pools: neither its outputs, its workspace nor its inputs may lie there."""
    meta = 2 * 2 * 64 * 4
    for kw in (dict(a2=pool), dict(q2=pool + POOL - 4), dict(l2=pool), dict(l2=pool - 4), dict(ws=pool), dict(ws=pool + POOL - 256),
               dict(ws=pool - 256), dict(a=pool), dict(a=pool - meta + 4), dict(q=pool + 4096), dict(ln=pool), dict(nxt=pool + POOL - 4),
               dict(a=pool, a2=pool), dict(q=pool, q2=pool), dict(ln=pool, l2=pool), dict(cache=pages(svx, table=pool + 64)),
               dict(cache=pages(svx, status=pool + POOL - 4))):
        assert refused(svx, evict(svx, **kw)), kw
    for kw in (dict(), dict(a2=pool + POOL), dict(l2=pool - 8), dict(ws=pool + POOL), dict(a=pool - meta), dict(a2=ACC, q2=POS, l2=LEN)):
        assert not refused(svx, evict(svx, **kw)), kw


def append(svx, cache=None, start=LEN, q_out=O, acc=ACC, pos=POS2, **kw):
    c, rope = cache or pages(svx), svx.Rope(128)
    return svx.lib.svx_paged_append(ctypes.byref(heads(svx, **kw)), ctypes.byref(rope.table), ctypes.byref(c), start, q_out, acc, pos, None)


@pytest.mark.parametrize("pool", [K, V], ids=["k", "v"])
def test_append_refuses_buffers_in_the_pools(svx, pool):
    inputs = 2 * (5 * 1024 + 512)
    for kw in (dict(pos=pool), dict(acc=pool + POOL - 4), dict(q_out=pool), dict(start=pool), dict(start=pool - 4), dict(q_norm=pool + 256),
               dict(k_norm=pool + POOL - 16), dict(n_new=pool), dict(q=pool), dict(k=pool + POOL - 16), dict(v=pool - 16),
               dict(cache=pages(svx, table=pool)), dict(cache=pages(svx, status=pool))):
        assert refused(svx, append(svx, **kw)), kw
    h = heads(svx, pos=pool + 1024)  # (the tokens' positions, an input)
    assert refused(svx, svx.lib.svx_paged_append(ctypes.byref(h), ctypes.byref(svx.Rope(128).table), ctypes.byref(pages(svx)), LEN, O, ACC, POS2,
                                                 None))
    for kw in (dict(), dict(start=pool + POOL), dict(start=pool - 8), dict(q_norm=pool - 256), dict(q=pool + POOL), dict(q=pool - inputs)):
        assert not refused(svx, append(svx, **kw)), kw


def test_pools_whose_rows_share_memory_are_refused_where_they_are_written(svx):
    """K and V may be interleaved in one tensor, in any way that keeps their rows apart; rows that coincide, in part or whole, of the two
    pools or of one, are refused by append and eviction.  One buffer read as both (decode) is fine, and so is moving its rows."""
    page, tok = 16 * 2 * 128, 2 * 128

    def both(**kw):
        c = pages(svx, **kw)
        a, e, r = append(svx, cache=c), evict(svx, cache=c), decode(svx, cache=c)
        return (a == svx.ERR_INVALID_ARG, e == svx.ERR_INVALID_ARG, r == svx.ERR_INVALID_ARG)
    apart = [dict(v=K + 2 * 128, head_stride=256, tok_stride=512, page_stride=16 * 512),          # [page][slot][head][K, V][d]
             dict(v=K + 2 * 2 * 128, tok_stride=512, page_stride=16 * 512),                        # [page][slot][K, V][head][d]
             dict(v=K + 2 * page, page_stride=2 * page),                                           # [page][K, V][slot][head][d]
             dict(v=K + 2 * 10 * page), dict(v=K - 2 * 10 * page),                                 # [K, V][page]..
             dict(v=K - 2 * page, page_stride=2 * page),                                           # V first
             dict(head_stride=16 * 128, tok_stride=128, v=K + 2 * page, page_stride=2 * page),     # heads outside the slots
             dict(page_stride=128, tok_stride=10 * 128, head_stride=16 * 10 * 128)]                # pages innermost
    for kw in apart:
        assert both(**kw) == (False, False, False), kw
    collide = [dict(v=K + 16), dict(v=K - 16), dict(v=K + 2 * 128 * 2), dict(v=K + 2 * page), dict(v=K + 2 * (9 * page)), dict(v=K + POOL - 16),
               dict(v=K - POOL + 16), dict(v=K + 2 * page - 16, page_stride=2 * page), dict(v=K + 2 * page + 16, page_stride=2 * page),
               dict(v=K + 2 * 128 + 16, head_stride=256, tok_stride=512, page_stride=16 * 512),
               dict(tok_stride=128), dict(page_stride=page - 8), dict(page_stride=tok), dict(head_stride=136, tok_stride=256)]
    for kw in collide:
        assert both(**kw) == (True, True, False), kw
    assert both(v=K) == (True, False, False)
    # against all pairs of rows, at small sizes
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(300):
        n = [rng.randint(1, 3) for _ in range(3)]
        s = [64 + 8 * rng.randrange(0, 60) for _ in range(3)]
        if rng.random() < 0.8:  # a nested layout, with gaps or without, in any order
            span, order = 64, rng.sample(range(3), 3)
            for i in order:
                s[i] = span + 8 * rng.choice([0, 0, 8, 24])
                span = s[i] * n[i]
        off = 8 * rng.randrange(-90, 90)
        kw = dict(v=K + 2 * off, n_pages=n[0], page_size=n[1], n_kv_heads=n[2], page_stride=s[0], tok_stride=s[1], head_stride=s[2], head_dim=64,
                  max_pages=4)
        begin = [a * s[0] + b * s[1] + c * s[2] for a in range(n[0]) for b in range(n[1]) for c in range(n[2])]
        own = any(abs(x - y) < 64 for i, x in enumerate(begin) for y in begin[:i])
        cross = off != 0 and any(abs(off + x - y) < 64 for x in begin for y in begin)
        got = evict(svx, cache=pages(svx, **kw)) == svx.ERR_INVALID_ARG
        if own or cross:
            assert got, kw
        nested, span = True, 64
        for stride, count in sorted((x, y) for x, y in zip(s, n) if y > 1):
            nested, span = nested and stride >= span, span + (count - 1) * stride
        if nested:  # (where strides do not nest, rows that happen to lie apart are refused too)
            assert got == cross, kw
        seen[got] += 1
    assert min(seen) > 40


def test_words_off_their_alignment_are_refused(svx):
    """int32 and fp32 buffers off the 4-byte grid (the kernels' loads and stores of them would be misaligned)."""
    def misaligned(status):
        return status == svx.ERR_INVALID_ARG and "aligned" in svx.lib.svx_last_error(None).decode()
    for by in (1, 2, 3):
        for kw in (dict(ln=LEN + by), dict(lse=LSE + by), dict(a=ACC + by), dict(b=ACC2 + by), dict(a=ACC + by, b=ACC + by)):
            assert misaligned(decode(svx, **kw)), kw
        for kw in (dict(ln=LEN + by), dict(nxt=NEXT + by), dict(a=ACC + by), dict(q=POS + by), dict(a2=ACC2 + by), dict(q2=POS2 + by),
                   dict(l2=LEN2 + by), dict(ln=LEN + by, l2=LEN + by)):
            assert misaligned(evict(svx, **kw)), kw
        for kw in (dict(start=LEN + by), dict(acc=ACC + by), dict(pos=POS2 + by), dict(n_new=NEXT + by)):
            assert misaligned(append(svx, **kw)), kw
        for kw in (dict(pos=POS + by), dict(n_new=NEXT + by), dict(status=STATUS + by)):
            h = heads(svx, **kw)
            assert misaligned(svx.lib.svx_qk_norm_rope(ctypes.byref(h), ctypes.byref(svx.Rope(128).table), O, K, V, None)), kw
            assert "status" in kw or misaligned(svx.lib.svx_paged_append(ctypes.byref(h), ctypes.byref(svx.Rope(128).table),
                                                                        ctypes.byref(pages(svx)), LEN, O, None, None, None)), kw


def test_scales_that_overflow_in_log2_units_are_refused(svx):
    """The kernel holds scores in log2 units: scale log2 e must be a finite fp32 number (an infinite one makes NaN of a score of 0)."""
    def status(scale):
        return refused(svx, decode(svx, scale=scale), words=("scale",))
    assert all(status(x) for x in (2.9e38, 2.4e38, 3.3e38, float("inf"), float("nan"), -1.0, -1e-45))
    assert not any(status(x) for x in (0.0, 1e-45, 0.125, 1e30, 2.3e38))


def test_split_in_32_bits_is_the_exact_split():
    """The kernels' begin(c) = c q + floor(c r / used + 0.001) with c r / used as an fp32 product by the rounded reciprocal: for every used <= 256,
    r < used and c <= used it is c q + (c r) // used."""
    import numpy as np
    f = np.float32
    for used in range(1, 257):
        per = f(1) / f(used)  # rounded to nearest
        c, r = np.meshgrid(np.arange(used + 1), np.arange(used), indexing="ij")
        cr = (c * r).astype(f)
        assert (cr == c * r).all()
        # one rounding: the product of two fp32 numbers is exact in fp64, and the sum keeps 2^-37 beside quotients below 256
        got = np.floor((cr.astype(np.float64) * float(per) + float(f(0.001))).astype(f))
        assert (got == (c * r) // used).all(), used


def test_streams_of_another_device_are_refused(svx, monkeypatch):
    """The call would run on the current stream of its tensors' device in place of the one that was asked for."""
    torch = pytest.importorskip("torch")

    class Stream:
        device_index = 1
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("current", s))
    with pytest.raises(svx.SvxError, match="cuda:1"):
        svx._on_stream(Stream(), 0)
    mine = Stream()
    assert svx._on_stream(mine, 1) == ("current", mine)
    q, pos = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.int32)
    for stream in (0, mine):  # tensors on the CPU, whatever the stream
        with pytest.raises(svx.SvxError):
            svx.qk_norm_rope(q, q, None, pos, svx.Rope(64), q, q, stream=stream)
