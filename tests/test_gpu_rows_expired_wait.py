"""A wait inside the kernel of many rows that runs out (svx_debug_expire_rows: one on a barrier on which nothing arrives, for a millisecond):
the kernel ends by itself, the rows that it had to do are NaN, whether or not there is a status word, and the next call is right."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

WAIT = 1  # the status word's bit


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


class Expire:
    def __init__(self, svx):
        self.svx = svx

    def __enter__(self):
        assert self.svx.lib.svx_debug_expire_rows(1) == self.svx.OK

    def __exit__(self, *_):
        assert self.svx.lib.svx_debug_expire_rows(0) == self.svx.OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b, n, states", [(3, 40, 1500), (1, 40, 20000), (3, 300, 1500), (1, 700, 9000), (160, 20, 1300)])
def test_states(svx, b, n, states, d):
    """Items that are split over CTAs and items that are not, of one row tile and of two."""
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((b, 2, n, d), (b, states, 1, d), (b, states, 1, d)))
    lens = torch.full((b,), states, dtype=torch.int32, device="cuda")
    lens[b // 2] = 0 if b > 1 else states
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, want_lse = torch.zeros_like(q), torch.zeros((b, 2, n), device="cuda")
    svx.cross_attn(q, k, v, want, want_lse, lens=lens, status=status)
    assert status.item() == 0 and not want.isnan().any()
    for word in (status, None):
        o, lse = torch.full_like(q, 7.0), torch.full((b, 2, n), 7.0, device="cuda")
        with Expire(svx):
            svx.cross_attn(q, k, v, o, lse, lens=lens, status=word)
        some = lens > 0
        assert o[some].isnan().all() and lse[some].isnan().all()
        assert (o[~some] == 0).all() and (lse[~some] == -math.inf).all()  # (no key: nothing to wait for)
        with Expire(svx):
            svx.cross_attn(q, k, v, o, None, lens=lens, status=word)
        assert o[some].isnan().all()
        svx.cross_attn(q, k, v, o, lse, lens=lens)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert status.item() == WAIT


@pytest.mark.parametrize("batch", [12, 100])
def test_prefixes(svx, batch):
    """Rows of a prefix are spoilt, those of requests without one are not."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    d, page = 128, 64
    k, v = (torch.randn((60, page, 2, d), generator=g, device="cuda").half() for _ in range(2))
    c = svx.PagedCache(k, v)
    q = torch.randn((batch + 3, 8, 1, d), generator=g, device="cuda").half()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    far = torch.arange(50, dtype=torch.int32, device="cuda")[None]
    table, lens = torch.full((batch + 3, 1), 55, dtype=torch.int32, device="cuda"), ints(*[i % 60 for i in range(batch + 3)])

    def run():
        o, lse = torch.full_like(q, 7.0), torch.full((batch + 3, 8, 1), 7.0, device="cuda")
        c.decode_shared(q, far, ints(3111), ints(0, batch), table, lens, o, lse)
        return o, lse

    want = run()
    assert not c.check()
    with Expire(svx):
        o, lse = run()
    assert o[:batch].isnan().all() and lse[:batch].isnan().all()
    assert torch.equal(o[batch:], want[0][batch:]) and torch.equal(lse[batch:], want[1][batch:])
    assert c.check()
    for x, y in zip(run(), want):
        assert torch.equal(x, y)
    assert not c.check()
