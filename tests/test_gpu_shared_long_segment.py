"""A prefix so long that a CTA's part of one item takes longer than the limit of a single wait."""
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


def test_a_segment_of_seconds(svx):
    """3 * 2^26 slots (in one page of an odd size that the table names over and over), 5 KV heads of one row tile each.  The tables of the
    requests' own slots have room for so many that the prefix has few CTAs (4), the first of them an item and a part of the next one, whose Q
    waits some 3 seconds for the first one's tiles (4 s in all).  Scores are 0, so that sums of weights are multiples of 128 (a tile's), exact up to 2^31:
    LSE = ln n.  (V is 0: this is about the wait.)"""
    n, page, d, heads, batch = 3 << 26, 8191, 128, 5, 17
    k = torch.ones((1, page, heads, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = svx.PagedCache(k, v)
    q = torch.zeros((batch, heads, 1, d), dtype=torch.bfloat16, device="cuda")
    far = torch.zeros((1, -(-n // page)), dtype=torch.int32, device="cuda")
    table = torch.zeros((batch, 278_000_000 // page), dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = torch.full_like(q, 7.0), torch.zeros((batch, heads, 1), device="cuda")
    args = q, far, ints(n), ints(0, batch), table, ints(*[0] * batch), o, lse
    c.decode_shared(*args)
    assert not c.check()
    assert (o == 0).all() and (lse.double() - math.log(n)).abs().max() < math.log(n) * 2.0 ** -22
