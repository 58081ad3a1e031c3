"""k and v of attention to an encoder's states that differ in the strides of dimensions of one entry, which nothing steps over
(bounds: attention_reference.near)."""
import pytest
import torch

from attention_reference import attend64, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


@pytest.mark.parametrize("n", [1, 24, 200])
@pytest.mark.parametrize("b, states, hkv", [(1, 300, 2), (2, 1, 2), (2, 300, 1), (1, 1, 1)])
def test_one_request_one_state_or_one_head(svx, b, states, hkv, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k = 2 * r(b, 2 * hkv, n, 64), r(b, states, hkv, 64)
    # the same strides, but for dimensions of one entry
    stride = [s + 8 * (i + 1) if size == 1 else s for i, (s, size) in enumerate(zip(k.stride()[:3], k.shape))]
    v = torch.as_strided(r(k.numel() + 4096), k.shape, (*stride, 1))
    assert v.stride() != k.stride()
    o, lse = torch.full_like(q, 7.0), torch.full((b, 2 * hkv, n), 7.0, device="cuda")
    svx.cross_attn(q, k, v, o, lse)
    for i in range(b):
        for h in range(hkv):
            x = slice(2 * h, 2 * h + 2)
            want = attend64(q[i, x].reshape(-1, 64), k[i, :, h], v[i, :, h], 64 ** -0.5)
            p_error = 2.0 ** -15 + (2.0 ** -8 if 2 * n > 128 else 0.0)  # (more than 128 rows: weights in bf16)
            near(o[i, x].reshape(-1, 64), lse[i, x].reshape(-1), want, p_error, states)


def test_other_strides_are_refused(svx):
    q = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((2, 50, 2, 64), dtype=torch.bfloat16, device="cuda")
    by_head = torch.zeros((2, 2, 50, 64), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    for v in (by_head, k[:, :49], k[:, :, :1]):
        with pytest.raises(svx.SvxError) as e:
            svx.cross_attn(q, k, v, torch.empty_like(q))
        assert e.value.status == svx.ERR_INVALID_ARG
