"""svx_residual_norm's checks of its arguments, without a GPU: addresses that are never followed."""
import ctypes

import pytest

BASE = 1 << 40  # (addresses only: every call here is refused, or fails because there is no such device)


@pytest.fixture(scope="module")
def svx():
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def args(svx, **change):
    gap = 1 << 24
    a = dict(h=BASE, y=BASE + gap, h_out=BASE + 2 * gap, x_out=BASE + 3 * gap, gate=None, norm=BASE + 4 * gap, post_norm=None,
             h_stride=64, y_stride=64, gate_stride=0, h_out_stride=64, x_stride=64, rows=100, dim=64, dtype=0, stream_dtype=0,
             gate_kind=0, act=0, device=0, alpha=1.0, beta=1.0, eps=1e-6, post_eps=-1.0, flags=1, pad=0)
    a.update(change)
    return svx.Residual(**a)


def call(svx, **change):
    return svx.lib.svx_residual_norm(ctypes.byref(args(svx, **change)), None)


@pytest.mark.parametrize("change", [
    dict(h=None), dict(h_out=None, x_out=None), dict(rows=0), dict(rows=1 << 31), dict(h_stride=60), dict(h_stride=-64),
    dict(h_out_stride=0), dict(x_stride=56), dict(h=BASE + 8), dict(norm=BASE + 2), dict(gate=BASE + (5 << 24)), dict(gate_kind=1),
    dict(gate_kind=4, gate=BASE + (5 << 24)), dict(act=1), dict(act=3, gate_kind=2, gate=BASE + (5 << 24)),
    dict(gate_kind=2, gate=BASE + (5 << 24) + 8), dict(gate_kind=1, gate=BASE + (5 << 24) + 1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(alpha=float("nan")), dict(beta=float("inf")), dict(post_eps=float("nan")), dict(post_norm=BASE + (5 << 24)),
    dict(x_out=None), dict(y=None, post_eps=0.0), dict(y=None, gate_kind=1, gate=BASE + (5 << 24)),
    # outputs over inputs and one another
    dict(h_out=BASE + 128, h_out_stride=64), dict(h_out=BASE, h_out_stride=128), dict(x_out=BASE), dict(h_out=BASE + (1 << 24)),
    dict(x_out=BASE + (2 << 24) + 64 * 2 * 99), dict(h_out=BASE + (4 << 24) - 64), dict(x_out=BASE + (1 << 24), x_stride=72),
    dict(stream_dtype=2, h_out=BASE + 64 * 4 * 99),
], ids=str)
def test_refused(svx, change):
    assert call(svx, **change) == svx.ERR_INVALID_ARG
    assert svx.lib.svx_last_error(None)


@pytest.mark.parametrize("change", [dict(dtype=2), dict(stream_dtype=1), dict(stream_dtype=3), dict(dim=4), dict(dim=60), dict(dim=16392)],
                         ids=str)
def test_unsupported(svx, change):
    assert call(svx, **change) == svx.ERR_UNSUPPORTED


def test_null(svx):
    assert svx.lib.svx_residual_norm(None, None) == svx.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(), dict(h_out=BASE), dict(x_out=BASE + (1 << 24)), dict(h_stride=0, y_stride=0), dict(stream_dtype=2, h_out=BASE + 64 * 4 * 100),
    dict(rows=1, h_out_stride=0, x_stride=3), dict(gate_kind=1, gate=BASE + (5 << 24) + 2), dict(x_out=None, norm=None, eps=-1.0),
    dict(y=None), dict(gate_kind=3, gate=BASE + (1 << 24), gate_stride=0),  # (a gate may be the block's output)
], ids=str)
def test_accepted_up_to_the_device(svx, change):
    """What the checks let through ends at the device: one that does not exist."""
    import torch
    device = torch.cuda.device_count() + 7
    assert call(svx, device=device, **change) == svx.ERR_CUDA
