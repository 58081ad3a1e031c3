"""The logarithm of a softmax's sum is the same whichever kernel takes the rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16], ids=str)
def test_the_same_sum_has_the_same_logarithm(svx, t, d):
    """1 to 512 of 2048 states, with a score of 0: sums of weights are the numbers of states (times a power of two), exact, so that LSE is the rounding
    of one and the same number, within log2f's ulp of log2(sum) times ln 2, and O = V = 1."""
    for base in (0, 256):
        lens = torch.arange(base + 1, base + 257, dtype=torch.int32, device="cuda")
        k = torch.ones((1, 2048, 1, d), dtype=t, device="cuda").expand(256, -1, 1, d)
        seen = {}
        for rows in (10, 20, 200):  # one block of 16 rows, one row tile, two
            q = torch.zeros((256, 1, rows, d), dtype=t, device="cuda")
            o, lse = torch.zeros_like(q), torch.zeros((256, 1, rows), device="cuda")
            svx.cross_attn(q, k, k, o, lse, lens=lens)
            assert (o == 1).all()
            assert (lse == lse[..., :1]).all()
            seen[rows] = lse[:, 0, 0].clone()
        assert torch.equal(seen[10], seen[20]) and torch.equal(seen[10], seen[200])
        want = torch.log(lens.double())
        lift = 7 if t == torch.float16 else 0  # (weights are held 2^7 times as large)
        ulp = 2.0 ** (torch.floor(torch.log2(lift + torch.log2(lens.double())).clamp(min=-30)) - 23)
        assert ((seen[10].double() - want).abs() <= ulp * 0.6932 + want * 2.0 ** -23).all()
