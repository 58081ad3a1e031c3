"""The residual stream between two blocks on the GPU against a plain 64-bit implementation.

Error bounds, derived before any run.  fp32 throughout, one rounding u = torch.finfo(type).eps / 2 at the end.  A mean of squares adds
at most 32 of a thread's terms in a row and 10 levels of a tree, each within 2^-24, and its square root and the division
stay under 2^-21: a norm is within 2^-18 of itself.  tanh and the sigmoid stay within 2^-19 (their arguments are 16-bit
values, here below 16), so the branch g u is within 2^-17 of itself and h' within e = 2^-22 |alpha h| + 2^-17 |beta g u| of its value.  The norm
of h' divides by its root mean square, which such errors move by |e| / |h'| at most (norms over the row), so x is within
2^-18 |x| + |norm| r e + |x| |e| / |h'|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def inputs(rows, dim, ty, stream, post, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    t, st = TYPES[ty], TYPES[stream]
    s = dict(h=(3 * torch.randn((rows, dim), generator=g)).to(st), y=torch.randn((rows, dim), generator=g).to(t),
             norm=(1 + 0.3 * torch.randn(dim, generator=g)).to(t), post_norm=None, gate=None)
    if post == "weights":
        s["post_norm"] = (1 + 0.3 * torch.randn(dim, generator=g)).to(t)
    shape = {"none": None, "scalar": (1,), "channel": (dim,), "element": (rows, dim)}[gate]
    if shape:
        s["gate"] = (2 * torch.randn(shape, generator=g)).to(t)
    s["y"][0] = 0  # a row whose norm is its eps alone
    return s


def reference(s, post, act, alpha, beta, eps=1e-6, post_eps=1e-5):
    """h', x and their error bounds before rounding."""
    h = s["h"].double() * alpha
    u = torch.zeros_like(h)
    if s["y"] is not None:
        u = s["y"].double()
        if post:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + post_eps)
            if s["post_norm"] is not None:
                u = u * s["post_norm"].double()
        if s["gate"] is not None:
            g = s["gate"].double()
            u = u * (torch.tanh(g) if act == "tanh" else torch.sigmoid(g) if act == "sigmoid" else g)
        u = u * beta
    z = h + u
    e = h.abs() * 2.0 ** -22 + u.abs() * 2.0 ** -17
    r = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
    w = 1.0 if s["norm"] is None else s["norm"].double()
    x = z * r * w
    size = torch.linalg.vector_norm(z, dim=-1, keepdim=True).clamp(min=1e-30)
    ex = x.abs() * 2.0 ** -18 + (z * 0 + w).abs() * r * e + x.abs() * torch.linalg.vector_norm(e, dim=-1, keepdim=True) / size
    return z, e, x, ex


def near(got, want, err):
    t = got.dtype
    bound = err + (want.abs() + err) * (torch.finfo(t).eps / 2) + torch.finfo(t).tiny * torch.finfo(t).eps
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), f"{float((off / bound).max()):.3f} times the bound"


def cuda(s):
    return {k: None if v is None else v.cuda() for k, v in s.items()}


CASES = [  # rows, dim, type, stream, norm after the block, gate, act, alpha, beta
    (1, 8, "bf16", "bf16", "", "none", None, 1.0, 1.0),
    (1, 4096, "bf16", "bf16", "", "scalar", "tanh", 1.0, 1.0),
    (3, 64, "fp16", "fp16", "weights", "channel", "sigmoid", 0.5, 2.0),
    (5, 256, "bf16", "fp32", "ones", "element", "tanh", 1.0, 0.25),
    (2, 264, "fp16", "fp32", "weights", "none", None, 1.25, -1.0),
    (7, 1024, "bf16", "bf16", "weights", "element", "sigmoid", 1.0, 1.0),
    (9, 1032, "fp16", "fp16", "ones", "channel", None, 0.9, 1.1),
    (33, 5128, "fp16", "fp32", "weights", "channel", "tanh", 1.0, 0.22),
    (2, 16384, "bf16", "fp32", "weights", "element", "tanh", 1.0, 1.0),
    (4, 16376, "bf16", "bf16", "", "element", None, 0.0, 1.0),
    (300, 2048, "bf16", "bf16", "weights", "scalar", "sigmoid", 1.0, 1.0),
    (1027, 128, "fp16", "fp16", "weights", "element", "tanh", 1.0, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_residual_norm(svx, case):
    rows, dim, ty, stream, post, gate, act, alpha, beta = case
    s = inputs(rows, dim, ty, stream, post, gate)
    z, e, x, ex = reference(s, post, act, alpha, beta)
    c = cuda(s)
    ho, xo = torch.full_like(c["h"], 7.0), torch.full_like(c["y"], 7.0)
    svx.residual_norm(c["h"], c["y"], ho, xo, norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5 if post else None,
                      gate=c["gate"], act=act, alpha=alpha, beta=beta)
    near(ho, z, e)
    near(xo, x, ex)
    assert torch.equal(c["h"].cpu(), s["h"]) and torch.equal(c["y"].cpu(), s["y"])


@pytest.mark.parametrize("dim", [72, 4096])
def test_in_place_alone_and_without_a_block(svx, dim):
    s = inputs(6, dim, "bf16", "bf16", "weights", "channel", seed=1)
    z, e, x, ex = reference(s, True, "tanh", 1.0, 0.5)
    c = cuda(s)
    kw = dict(norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5, gate=c["gate"], act="tanh", beta=0.5)
    ho, xo = torch.empty_like(c["h"]), torch.empty_like(c["y"])
    svx.residual_norm(c["h"], c["y"], ho, xo, **kw)
    only_h, only_x = torch.empty_like(ho), torch.empty_like(xo)
    svx.residual_norm(c["h"], c["y"], only_h, None, **{**kw, "norm": None})
    svx.residual_norm(c["h"], c["y"], None, only_x, **kw)
    assert torch.equal(only_h, ho) and torch.equal(only_x, xo)
    svx.residual_norm(c["h"], c["y"], c["h"], c["y"], **kw)  # both in place
    assert torch.equal(c["h"], ho) and torch.equal(c["y"], xo)
    near(ho, z, e)
    near(xo, x, ex)
    s2 = inputs(6, dim, "fp16", "fp32", "", "none", seed=2)
    s2["y"] = None
    z, e, x, ex = reference(s2, False, None, 0.5, 1.0)
    xo = torch.empty((6, dim), dtype=torch.float16, device="cuda")
    svx.residual_norm(s2["h"].cuda(), None, None, xo, norm=s2["norm"].cuda(), alpha=0.5)
    near(xo, x, ex)


def test_strided_rows_and_leading_dimensions(svx):
    """Slices of wider buffers, broadcast inputs, three leading shapes; what lies between the rows stays."""
    b, n, dim = 3, 5, 320
    s = inputs(b * n, dim, "bf16", "bf16", "weights", "element", seed=3)
    z, e, x, ex = reference(s, True, "sigmoid", 1.0, 1.0)
    wide = {k: torch.full((b, n, dim + 40), 9.0, dtype=torch.bfloat16, device="cuda") for k in ("h", "y", "gate", "ho", "xo")}
    view = {k: w[..., 16:16 + dim] for k, w in wide.items()}
    for k in ("h", "y", "gate"):
        view[k].copy_(s[k].reshape(b, n, dim))
    svx.residual_norm(view["h"], view["y"], view["ho"], view["xo"], norm=s["norm"].cuda(), post_norm=s["post_norm"].cuda(),
                      post_eps=1e-5, gate=view["gate"], act="sigmoid")
    near(view["ho"].reshape(b * n, dim), z, e)
    near(view["xo"].reshape(b * n, dim), x, ex)
    for k in ("ho", "xo"):
        assert (wide[k][..., :16] == 9).all() and (wide[k][..., 16 + dim:] == 9).all()
    row = s["h"][:1].cuda()
    s["h"] = s["h"][:1].expand(b * n, dim)
    xo = torch.empty((b * n, dim), dtype=torch.bfloat16, device="cuda")
    svx.residual_norm(row.expand(b * n, dim), s["y"].cuda(), None, xo, norm=s["norm"].cuda(), gate=s["gate"].cuda())
    z, e, x, ex = reference(s, False, None, 1.0, 1.0)
    near(xo, x, ex)


def test_values_that_are_not_finite_stay_in_their_row(svx):
    s = inputs(4, 1536, "bf16", "bf16", "weights", "none", seed=4)
    z, e, x, ex = reference(s, True, None, 1.0, 1.0)
    c = cuda(s)
    c["y"][1, 7], c["h"][2, 3] = float("nan"), float("inf")
    ho, xo = torch.empty_like(c["h"]), torch.empty_like(c["y"])
    svx.residual_norm(c["h"], c["y"], ho, xo, norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5)
    keep = [0, 3]
    near(ho[keep], z[keep], e[keep])
    near(xo[keep], x[keep], ex[keep])
    assert xo[1].isnan().all() and xo[2, 3].isnan()


def test_streams_and_graphs(svx):
    s = inputs(40, 1024, "bf16", "fp32", "weights", "channel", seed=5)
    c = cuda(s)
    want_h, want_x = torch.empty_like(c["h"]), torch.empty_like(c["y"])
    kw = dict(norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5, gate=c["gate"], act="tanh")
    svx.residual_norm(c["h"], c["y"], want_h, want_x, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ho, xo = torch.zeros_like(want_h), torch.zeros_like(want_x)
    svx.residual_norm(c["h"], c["y"], ho, xo, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ho, want_h) and torch.equal(xo, want_x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svx.residual_norm(c["h"], c["y"], ho, xo, **kw)
        svx.residual_norm(ho, xo, c["h"], c["y"], norm=c["norm"])
    ho.zero_()
    xo.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ho, want_h) and torch.equal(xo, want_x)


def test_refusals(svx):
    h = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    y, ho, xo = (torch.zeros_like(h) for _ in range(3))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    bad = [
        (dict(y=y.half()), svx.ERR_UNSUPPORTED), (dict(y=y.float()), svx.ERR_UNSUPPORTED), (dict(y=y[:3]), svx.ERR_INVALID_ARG),
        (dict(x_out=xo.float()), svx.ERR_INVALID_ARG), (dict(h_out=ho.float()), svx.ERR_INVALID_ARG),
        (dict(h_out=None, x_out=None), svx.ERR_INVALID_ARG), (dict(h_out=y), svx.ERR_INVALID_ARG),
        (dict(x_out=h), svx.ERR_INVALID_ARG), (dict(x_out=ho), svx.ERR_INVALID_ARG), (dict(norm=w[:32]), svx.ERR_INVALID_ARG),
        (dict(norm=w.float()), svx.ERR_INVALID_ARG), (dict(gate=w[:32]), svx.ERR_INVALID_ARG), (dict(gate=y[:2]), svx.ERR_INVALID_ARG),
        (dict(act="tanh"), svx.ERR_INVALID_ARG), (dict(gate=w, act="relu"), svx.ERR_INVALID_ARG), (dict(post_norm=w), svx.ERR_INVALID_ARG),
        (dict(post_eps=-1.0), svx.ERR_INVALID_ARG), (dict(eps=-1.0), svx.ERR_INVALID_ARG), (dict(eps=float("nan")), svx.ERR_INVALID_ARG),
        (dict(alpha=float("inf")), svx.ERR_INVALID_ARG), (dict(y=None, gate=w), svx.ERR_INVALID_ARG),
        (dict(y=None, post_eps=1e-6), svx.ERR_INVALID_ARG), (dict(norm=w, x_out=None), svx.ERR_INVALID_ARG),
        (dict(y=y.cpu()), svx.ERR_INVALID_ARG), (dict(x_out=xo[0].expand(4, 64)), svx.ERR_INVALID_ARG),
    ]
    for change, status in bad:
        kw = dict(h=h, y=y, h_out=ho, x_out=xo)
        kw.update(change)
        with pytest.raises(svx.SvxError) as e:
            svx.residual_norm(**kw)
        assert e.value.status == status, (change.keys(), e.value)
    for dim in (12, 16392):  # not a multiple of 8, too long
        big = torch.zeros((2, dim), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(svx.SvxError) as e:
            svx.residual_norm(big, None, None, torch.empty_like(big))
        assert e.value.status == svx.ERR_UNSUPPORTED
    odd = torch.zeros(4 * 72 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(4, 72)[:, :64]  # 8 bytes off the 16-byte grid
    with pytest.raises(svx.SvxError):
        svx.residual_norm(odd, y, ho, xo)
    uneven = torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16, device="cuda")[:, ::2, :2]
    with pytest.raises(svx.SvxError):
        svx.residual_norm(uneven, None, None, torch.empty((2, 2, 2, 64), dtype=torch.bfloat16, device="cuda"))
