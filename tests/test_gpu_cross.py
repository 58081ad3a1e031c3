"""Attention to an encoder's states on the GPU against a plain 64-bit implementation (bounds: attention_reference.near).

With up to 128 rows (query heads of a KV head times tokens) a softmax weight enters the product with V in two 16-bit pieces, within 2^-15 of
itself with its exponential and its sum; with more it is rounded to the inputs' type once, by half a step."""
import pytest
import torch

from attention_reference import attend64, near

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def p_error(rows, ty):
    return 2.0 ** -15 + (torch.finfo(TYPES[ty]).eps / 2 if rows > 128 else 0.0)


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def inputs(b, n, hq, hkv, d, states, ty, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[ty]
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    if layout == "fused":
        kv = r(b, states, 2, hkv, d)
        k, v = kv[:, :, 0], kv[:, :, 1]
        q, o = 2 * r(b, n, hq, d).transpose(1, 2), torch.full((b, n, hq, d), 7.0, dtype=t, device="cuda").transpose(1, 2)
    else:
        k, v = r(b, hkv, states, d).transpose(1, 2), r(b, hkv, states, d).transpose(1, 2)
        q, o = 2 * r(b, hq, n, d), torch.full((b, hq, n, d), 7.0, dtype=t, device="cuda")
    return q, k, v, o, torch.full((b, hq, n), 7.0, device="cuda")


def visible(b, states, lens, mask):
    live = torch.ones((b, states), dtype=torch.bool, device="cuda")
    if lens is not None:
        live &= torch.arange(states, device="cuda")[None, :] < lens[:, None].clamp(0, states)
    if mask is not None:
        live &= mask
    return live


def check(q, k, v, o, lse, live, ty, scale=None):
    b, hq, n, d = q.shape
    hkv = k.shape[2]
    group = hq // hkv
    for i in range(b):
        at = live[i].nonzero()[:, 0]
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            want = attend64(q[i, heads].reshape(-1, d), k[i, at, h], v[i, at, h], scale or d ** -0.5)
            near(o[i, heads].reshape(-1, d), lse[i, heads].reshape(-1), want, p_error(group * n, ty), len(at))


CASES = [  # b, n, hq, hkv, d, states, type, layout, lens, masked
    (1, 1, 1, 1, 64, 1, "bf16", "fused", None, 0),
    (1, 1, 16, 16, 64, 1500, "fp16", "fused", None, 0),
    (2, 1, 8, 2, 128, 333, "bf16", "heads", (0, 333), 0.3),
    (3, 1, 28, 4, 128, 129, "fp16", "fused", (1, 128, 129), 0),
    (4, 5, 8, 2, 128, 700, "bf16", "fused", (700, 0, 1, 513), 0.5),      # 20 rows
    (2, 3, 6, 2, 64, 257, "fp16", "heads", None, 0.2),                    # 9 rows
    (1, 32, 4, 1, 64, 640, "bf16", "fused", None, 0),                     # 128 rows
    (1, 129, 1, 1, 128, 127, "fp16", "heads", None, 0),                   # 129 rows
    (2, 100, 3, 1, 128, 1000, "bf16", "fused", (1000, 63), 0.4),          # 300 rows
    (1, 77, 16, 2, 64, 2049, "fp16", "fused", None, 0.1),                 # 616 rows
    (5, 511, 2, 2, 64, 77, "bf16", "heads", (77, 20, 0, 1, 64), 0),
    (1, 700, 8, 8, 128, 3001, "bf16", "fused", None, 0),
    (64, 2, 2, 1, 64, 50, "bf16", "fused", None, 0.5),
    (256, 1, 2, 1, 64, 9, "fp16", "heads", tuple(i % 10 for i in range(256)), 0),
    (1, 1, 40, 1, 64, 1, "bf16", "fused", None, 0),                       # 40 heads to a KV head
    (1, 2, 4, 1, 128, 70000, "bf16", "fused", None, 0),
    (1, 300, 1, 1, 128, 40000, "fp16", "fused", None, 0.01),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_cross(svx, case):
    b, n, hq, hkv, d, states, ty, layout, lens, masked = case
    q, k, v, o, lse = inputs(b, n, hq, hkv, d, states, ty, layout)
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    mask = torch.rand((b, states), generator=g, device="cuda") >= masked if masked else None
    live = visible(b, states, lens, mask)
    k[~live], v[~live] = float("nan"), float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    svx.cross_attn(q, k, v, o, lse, lens=lens, mask=mask, status=status)
    check(q, k, v, o, lse, live, ty)
    assert status.item() == 0
    again = torch.full_like(o, 5.0)
    svx.cross_attn(q, k, v, again, None, lens=lens, mask=mask)  # no LSE, and the same result
    assert torch.equal(again, o)


@pytest.mark.parametrize("n", [1, 40])
def test_masks_that_leave_nothing_and_masks_at_the_ends(svx, n):
    """Requests whose mask leaves none, the first state, the last one, every other one; whole tiles hidden before and between."""
    states = 900
    q, k, v, o, lse = inputs(6, n, 4, 2, 128, states, "bf16", "fused", seed=2)
    mask = torch.zeros((6, states), dtype=torch.bool, device="cuda")
    mask[1, 0] = mask[2, -1] = True
    mask[3, ::2] = True
    mask[4, 640:700] = True
    mask[5] = True
    mask[5, 128:512] = False
    k[~mask], v[~mask] = float("nan"), float("nan")
    svx.cross_attn(q, k, v, o, lse, mask=mask)
    check(q, k, v, o, lse, mask, "bf16")
    assert (o[0] == 0).all() and (lse[0] == float("-inf")).all()
    svx.cross_attn(q, k[:, :1], v[:, :1], o, lse, mask=mask[:, :1])  # a mask with rows apart, one state
    check(q, k[:, :1], v[:, :1], o, lse, mask[:, :1], "bf16")


@pytest.mark.parametrize("n", [1, 200])
def test_no_states(svx, n):
    q, k, v, o, lse = inputs(2, n, 4, 2, 64, 5, "fp16", "fused")
    svx.cross_attn(q, k[:, :0], v[:, :0], o, lse)
    assert (o == 0).all() and (lse == float("-inf")).all()
    o.fill_(3)
    svx.cross_attn(q, k, v, o, lse, lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert (o == 0).all() and (lse == float("-inf")).all()


def test_lengths_out_of_bounds_are_clamped_and_reported(svx):
    for n in (1, 50):
        q, k, v, o, lse = inputs(3, n, 4, 2, 64, 200, "bf16", "heads", seed=3)
        lens = torch.tensor([-4, 100, 1000], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        svx.cross_attn(q, k, v, o, lse, lens=lens, status=status)
        check(q, k, v, o, lse, visible(3, 200, lens, None), "bf16")
        assert status.item() != 0


@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("ty", ["bf16", "fp16"])
def test_broadcast_states_scales_and_sharp_softmax(svx, n, ty):
    """One request's states for all of them (stride 0); a scale; scores of very unequal size, rising and falling along the states."""
    q, k, v, o, lse = inputs(4, n, 4, 2, 128, 1100, ty, "fused", seed=4)
    ramp = torch.linspace(-12, 12, 1100, device="cuda").to(k.dtype)
    for sign in (1, -1):
        kk = k.clone()
        kk[..., 0] = sign * ramp[None, :, None]
        one = (x[:1].expand(4, -1, -1, -1) for x in (kk, v.clone()))
        kk, vv = one
        svx.cross_attn(q, kk, vv, o, lse, scale=1.0)
        check(q, kk, vv, o, lse, visible(4, 1100, None, None), ty, scale=1.0)
    zero = torch.zeros_like(q)
    svx.cross_attn(zero, k, v, o, lse)  # equal weights
    check(zero, k, v, o, lse, visible(4, 1100, None, None), ty)


def test_samples_of_one_input_as_tokens(svx):
    """8 samples over one encoded input, one token each, as 8 tokens of it: the same as 8 requests."""
    q, k, v, o, lse = inputs(1, 8, 16, 4, 64, 600, "bf16", "heads", seed=5)
    svx.cross_attn(q, k, v, o, lse)
    check(q, k, v, o, lse, visible(1, 600, None, None), "bf16")
    flat = q[0].transpose(0, 1).contiguous()  # [sample][head][d]
    out = torch.empty_like(flat)
    svx.cross_attn(flat.transpose(0, 1)[None], k, v, out.transpose(0, 1)[None], None)
    assert torch.equal(out.transpose(0, 1)[None], o)


def test_what_lies_between_the_rows_stays(svx):
    for n in (2, 60):
        q, k, v, _, lse = inputs(2, n, 4, 2, 64, 300, "fp16", "fused", seed=6)
        wide = torch.full((2, n, 4, 3, 64), 9.0, dtype=torch.float16, device="cuda")
        o = wide[:, :, :, 1].transpose(1, 2)
        svx.cross_attn(q, k, v, o, lse)
        check(q, k, v, o, lse, visible(2, 300, None, None), "fp16")
        assert (wide[:, :, :, 0] == 9).all() and (wide[:, :, :, 2] == 9).all()


@pytest.mark.parametrize("n", [1, 150])
def test_graphs_streams_and_lengths_that_change(svx, n):
    q, k, v, o, lse = inputs(3, n, 8, 2, 128, 1000, "bf16", "fused", seed=7)
    lens = torch.tensor([10, 1000, 500], dtype=torch.int32, device="cuda")
    svx.cross_attn(q, k, v, o, lse, lens=lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svx.cross_attn(q, k, v, o, lse, lens=lens)
    for change in ([0, 1, 999], [1000, 1000, 1000], [128, 129, 0]):
        lens.copy_(torch.tensor(change))
        o.fill_(3)
        graph.replay()
        check(q, k, v, o, lse, visible(3, 1000, lens, None), "bf16")
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.empty_like(o), torch.empty_like(o)
    for _ in range(10):  # two calls at once
        svx.cross_attn(q, k, v, a, None, lens=lens, stream=side)
        svx.cross_attn(q, k, v, b, None, lens=lens, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(b, o)


def test_refusals(svx):
    q, k, v, o, lse = inputs(2, 3, 4, 2, 64, 100, "bf16", "fused")
    lens, mask = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones((2, 100), dtype=torch.bool, device="cuda")
    bad = [
        dict(q=q.float()), dict(k=k.half()), dict(v=v.contiguous()), dict(k=k[:1], v=v[:1]), dict(k=k[..., :32], v=v[..., :32]),
        dict(o=o[:, :, :2]), dict(o=o.float()), dict(lse=lse.half()), dict(lse=lse[:, :2]), dict(lens=lens.long()), dict(lens=lens[:1]),
        dict(mask=mask.float()), dict(mask=mask[:, :50]), dict(mask=mask.t().contiguous().t()), dict(q=q.cpu()), dict(o=q),
        dict(o=o[:, :1].expand(2, 4, 3, 64)), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=3.4e38),
        dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(k=k[:, :, :0], v=v[:, :, :0]),
        dict(q=q[..., 1:], k=k[..., 1:], v=v[..., 1:], o=o[..., 1:]), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")),
        dict(q=q[:, :3], o=o[:, :3], lse=lse[:, :3]),  # 3 query heads, 2 KV heads
        dict(q=torch.zeros((257, 4, 1, 64), dtype=q.dtype, device="cuda"), k=k[:1].expand(257, -1, -1, -1), v=v[:1].expand(257, -1, -1, -1),
             o=torch.zeros((257, 4, 1, 64), dtype=q.dtype, device="cuda"), lse=None),
    ]
    for change in bad:
        kw = dict(q=q, k=k, v=v, o=o, lse=lse)
        kw.update(change)
        with pytest.raises(svx.SvxError):
            svx.cross_attn(**kw)
    d32 = [torch.zeros((1, 2, 2, 32), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    with pytest.raises(svx.SvxError) as e:
        svx.cross_attn(*d32)
    assert e.value.status == svx.ERR_UNSUPPORTED
