"""residual_norm of a layer whose gate is optional, on the GPU: without a gate every activation leaves the results alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


@pytest.mark.parametrize("post_eps", [None, 1e-6])
@pytest.mark.parametrize("rows, dim, stream", [(1, 64, torch.bfloat16), (37, 520, torch.float32), (5, 4096, torch.bfloat16)])
def test_no_gate_and_any_activation(svx, rows, dim, stream, post_eps):
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda t: torch.randn((rows, dim), generator=g, device="cuda").to(t)  # noqa: E731
    h, y = r(stream), r(torch.bfloat16)
    norm = r(torch.bfloat16)[0].clone()
    out = {}
    for act in (None, "tanh", "sigmoid"):
        ho, xo = torch.full_like(h, 7.0), torch.full_like(y, 7.0)
        svx.residual_norm(h, y, ho, xo, norm=norm, post_eps=post_eps, gate=None, act=act, alpha=0.75, beta=1.25)
        out[act] = ho, xo
    ho, xo = torch.full_like(h, 5.0), torch.full_like(y, 5.0)
    svx.residual_norm(h, y, ho, xo, norm=norm, post_eps=post_eps, alpha=0.75, beta=1.25)
    for act, (a, b) in out.items():
        assert torch.equal(a, ho) and torch.equal(b, xo), act
    # one row by hand, in 64 bits: alpha h + beta u, rounded once (fp32 sums: 2^-20 of the terms)
    u = y[0].double()
    if post_eps is not None:
        u = u / torch.sqrt((u * u).mean() + post_eps)
    want, size = 0.75 * h[0].double() + 1.25 * u, h[0].double().abs() + 2 * u.abs()
    eps = torch.finfo(stream).eps / 2
    assert ((ho[0].double() - want).abs() <= want.abs() * eps + size * 2.0 ** -20).all()


def test_an_activation_where_no_gate_is_passed_is_refused(svx):
    h = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(svx.SvxError) as e:
        svx.residual_norm(h, torch.zeros_like(h), torch.zeros_like(h), act="tanh")
    assert e.value.status == svx.ERR_INVALID_ARG
