"""A prefix whose last tile ends at 2^31 slots: what lies behind its length does not count there either."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def test_a_prefix_of_almost_two_to_the_31_slots(svx):
    """2^31 - 8 slots, all of them in one page that the table names over and over, every key with a score of -30: LSE = ln(2^31 - 8) - 30.
    Eight slots behind the length with a score of 0 would be e^30 times as heavy each.  O is V, 1.0 in every row: weights and their
    sums are whole numbers below 2^24 in each CTA, so only the factors of the merge round."""
    page, pages, d, hq, batch = 38872, 55245, 64, 4, 8
    length = page * pages
    assert length == 2 ** 31 - 8
    k = torch.ones((2, page, 1, d), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    c = svx.PagedCache(k, v)
    q = torch.full((batch, hq, 1, d), -3.75, dtype=torch.bfloat16, device="cuda")  # q.k / 8 = -30
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    far, table = torch.zeros((1, pages), dtype=torch.int32, device="cuda"), torch.ones((batch, 1), dtype=torch.int32, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros((batch, hq, 1), device="cuda")
    for n in (length, length - 120, 1000):
        c.decode_shared(q, far, ints(n), ints(0, batch), table, ints(*[0] * batch), o, lse, max_len=1)
        assert (o == 1).all(), o.float().mean()
        want = math.log(n) - 30
        assert (lse.double() - want).abs().max() <= 30 * 2.0 ** -19 + 2.0 ** -19  # (a score's error, as everywhere; the merge's)
    assert not c.check()
