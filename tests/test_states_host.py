"""svx_cross_attn and svx_paged_decode_shared without a GPU: every refusal that comes before the first CUDA call (fake addresses,
which no call may follow), and what is let through up to the device."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def svx():
    from speculative_decoding_verification_chunked_gb300 import build
    if not all(os.path.exists(x) for x in (build.LIB, build.LIB_CHECKED, build.LIB_TORCH)):
        build.build()
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


# 256-byte aligned, far apart
Q, K, V, O, LSE, LEN, MASK, STATUS, WS, TABLE, FAR, FARLEN, FIRST = (0x100000000 * (i + 1) for i in range(13))


def cross(svx, **kw):
    """2 requests of 3 tokens, 4 heads and 2 KV heads of 64, 100 states, as fused projections leave them."""
    f = dict(q=Q, k=K, v=V, o=O, lse=LSE, len=LEN, mask=MASK, status=STATUS, q_req=3 * 256, q_head=64, q_tok=256, kv_req=100 * 256,
             kv_head=64, kv_state=256, o_req=3 * 256, o_head=64, o_tok=256, mask_req=100, n_req=2, n_tok=3, n_states=100, n_q_heads=4,
             n_kv_heads=2, head_dim=64, dtype=0, device=0, scale=0.0, flags=1)
    f.update(kw)
    return svx.Cross(*[f[n] for n, _ in svx.Cross._fields_])


def call_cross(svx, ws=WS, ws_bytes=1 << 40, **kw):
    return svx.lib.svx_cross_attn(ctypes.byref(cross(svx, **kw)), ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=Q + 8), dict(o=O + 2), dict(k=K + 4), dict(v=V + 8), dict(lse=LSE + 2),
    dict(len=LEN + 1), dict(status=STATUS + 2), dict(n_req=0), dict(n_req=257), dict(n_tok=0), dict(n_states=-1), dict(n_states=2 ** 31 - 1),
    dict(n_kv_heads=0), dict(n_q_heads=3), dict(n_q_heads=1, n_kv_heads=2), dict(n_q_heads=4100, n_kv_heads=2), dict(q_req=100),
    dict(q_head=-64), dict(q_tok=4), dict(kv_req=12), dict(kv_head=-8), dict(kv_state=1 << 45), dict(o_tok=0), dict(o_head=0),
    dict(o_req=64), dict(o_head=32), dict(mask_req=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=3e38),
    # outputs over inputs and one another
    dict(o=Q), dict(o=K + 256), dict(lse=V), dict(o=LSE), dict(status=LSE + 8), dict(lse=LEN), dict(lse=MASK + 100), dict(status=Q + 64),
], ids=str)
def test_cross_refuses(svx, kw):
    assert call_cross(svx, **kw) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_last_error(None)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(dtype=-1), dict(head_dim=96), dict(head_dim=256),
                                dict(n_req=1, n_tok=1 << 20), dict(n_req=200, n_tok=100000, n_states=1 << 22, q_req=0, o_req=1 << 30)],
                         ids=str)
def test_cross_does_not_support(svx, kw):
    assert call_cross(svx, **kw) == svx.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(), dict(lse=None, len=None, mask=None, status=None), dict(n_states=0, k=None, v=None), dict(k=V, v=V),
                                dict(q_req=0, q_head=0, q_tok=0, kv_req=0, kv_head=0, kv_state=0, mask_req=0), dict(n_req=1, n_tok=70000),
                                dict(n_req=1, q_req=3, kv_req=5, o_req=7), dict(mask=MASK + 3, mask_req=101), dict(o_req=64 * 7, o_head=64 * 14, o_tok=64)],
                         ids=str)
def test_cross_goes_to_the_device(svx, kw):
    """One that is not there."""
    import torch
    assert call_cross(svx, device=torch.cuda.device_count() + 9, **kw) == svx.ERR_CUDA


def test_null(svx):
    n = ctypes.c_int64()
    assert svx.lib.svx_cross_attn(None, WS, 1 << 30, None) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_cross_attn_workspace(None, ctypes.byref(n)) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_cross_attn_workspace(ctypes.byref(cross(svx)), None) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_paged_decode_shared_workspace(ctypes.byref(pages(svx)), 2, 4, None, 0, ctypes.byref(n)) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_paged_decode_shared_workspace(None, 2, 4, ctypes.byref(prefixes(svx)), 0, ctypes.byref(n)) == svx.ERR_INVALID_ARG


def pages(svx, **kw):
    f = dict(k=K, v=V, table=TABLE, status=STATUS, page_stride=16 * 2 * 128, tok_stride=2 * 128, head_stride=128, n_pages=10,
             page_size=16, max_pages=4, n_kv_heads=2, head_dim=128, dtype=0, device=0, flags=1, pad=0)
    f.update(kw)
    return svx.Pages(*[f[n] for n, _ in svx.Pages._fields_])


def prefixes(svx, **kw):
    f = dict(table=FAR, len=FARLEN, first=FIRST, max_len=0, n_prefix=2, max_pages=5)
    f.update(kw)
    return svx.Prefixes(*[f[n] for n, _ in svx.Prefixes._fields_])


def call_shared(svx, n_req=3, n_q=4, q=Q, len_=LEN, max_len=0, scale=0.0, o=O, lse=LSE, ws=WS, pages_=None, prefixes_=None):
    return svx.lib.svx_paged_decode_shared(ctypes.byref(pages(svx, **(pages_ or {}))), n_req, n_q, q, ctypes.byref(prefixes(svx, **(prefixes_ or {}))),
                                           len_, max_len, scale, o, lse, ws, 1 << 40, None)


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=257), dict(n_q=3), dict(n_q=0), dict(n_q=4098), dict(q=None), dict(q=Q + 8), dict(len_=None), dict(len_=LEN + 2),
    dict(o=None), dict(o=O + 4), dict(lse=None), dict(lse=LSE + 1), dict(max_len=-1), dict(max_len=65), dict(scale=-0.5), dict(scale=float("nan")),
    dict(prefixes_=dict(table=None)), dict(prefixes_=dict(len=None)), dict(prefixes_=dict(first=None)), dict(prefixes_=dict(first=FIRST + 2)),
    dict(prefixes_=dict(n_prefix=0)), dict(prefixes_=dict(n_prefix=257)), dict(prefixes_=dict(max_pages=0)),
    dict(prefixes_=dict(max_pages=1 << 28)), dict(prefixes_=dict(max_len=-1)), dict(prefixes_=dict(max_len=81)),
    dict(pages_=dict(k=None)), dict(pages_=dict(page_size=0)), dict(pages_=dict(tok_stride=4)),
    # outputs over inputs, the pools and one another
    dict(o=Q), dict(o=K + 512), dict(lse=V), dict(o=LSE), dict(lse=LEN), dict(lse=TABLE + 8), dict(lse=FAR + 36), dict(lse=FARLEN + 4),
    dict(lse=FIRST + 8), dict(pages_=dict(status=LSE + 4)), dict(pages_=dict(status=FIRST)),
], ids=str)
def test_shared_refuses(svx, kw):
    assert call_shared(svx, **kw) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_last_error(None)


@pytest.mark.parametrize("kw", [dict(), dict(max_len=64, prefixes_=dict(max_len=80)), dict(prefixes_=dict(n_prefix=256)), dict(n_req=256, n_q=32),
                                dict(prefixes_=dict(table=TABLE)), dict(pages_=dict(v=K))], ids=str)
def test_shared_goes_to_the_device(svx, kw):
    import torch
    kw = {**kw, "pages_": {**kw.get("pages_", {}), "device": torch.cuda.device_count() + 9}}
    assert call_shared(svx, **kw) == svx.ERR_CUDA


def test_the_even_split_in_float_is_exact():
    """begin(c) = c q + floor(c r / used): the kernels take the quotient from a float product with 1 / used, plus 0.001, rounded once."""
    import numpy as np
    for used in range(1, 257):
        p = np.arange(0, used + 1)[:, None] * np.arange(0, used)[None, :]
        x = p.astype(np.float64) * np.float64(np.float32(1) / np.float32(used)) + np.float64(np.float32(0.001))
        assert (np.floor(x.astype(np.float32)) == p // used).all(), used


def test_the_row_of_an_item_by_its_group_in_float_is_exact():
    """x / n from a float product with 1 / n, corrected by one: for every group up to 4096, around every multiple below 2^20."""
    import numpy as np
    for n in list(range(1, 200)) + [255, 256, 257, 511, 1000, 4095, 4096]:
        m = np.arange(0, (1 << 20) // n + 1, max(1, (1 << 20) // n // 4000), dtype=np.int64) * n
        for x in (m, m[m > 0] - 1, m + n - 1):
            q = (x.astype(np.float32) * (np.float32(1) / np.float32(n))).astype(np.int64)
            left = x - q * n
            q = np.where(left < 0, q - 1, np.where(left >= n, q + 1, q))
            assert (q == x // n).all(), n
