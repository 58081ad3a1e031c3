"""Many rows against millions of keys with V of one sign: products that are small beside their sum have to count all the same.

Bounds.  O: its rounding, half a step u; that of P (u again with more than 128 rows, else 2^-15 with its exponential and sum); what the tensor
cores leave out of at most 32768 products in a row, each less than 2^-24 of their sum: 2^-9.  LSE: a score's error 2^-19 S as everywhere (S up
to 8 here), a fp32 sum of `tiles` terms that grow with it, tiles 2^-24 at worst."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def attend64(q, k, v, scale):
    """Rows in 64 bits, some keys at a time: O and LSE."""
    top, total, o = (torch.zeros((len(q), n), dtype=torch.float64, device="cuda") for n in (1, 1, v.shape[1]))
    top -= math.inf
    for i in range(0, len(k), 1 << 18):
        s = q.double() @ k[i:i + (1 << 18)].double().T * scale
        m = torch.maximum(top, s.amax(-1, keepdim=True))
        p, back = torch.exp(s - m), torch.exp(top - m)
        total, o, top = total * back + p.sum(-1, keepdim=True), o * back + p @ v[i:i + (1 << 18)].double(), m
    return o / total, (top + torch.log(total))[:, 0]


def near(o, lse, want, p_error, tiles):
    wo, wl = want
    bound = wo.abs() * (torch.finfo(o.dtype).eps / 2 + 2 * p_error + 2.0 ** -9)
    off = (o.double() - wo).abs()
    assert (off <= bound).all(), f"o: {float((off / bound).max()):.3f} times the bound"
    assert ((lse.double() - wl).abs() <= 2.0 ** -15 + wl.abs() * 2.0 ** -22 + tiles * 2.0 ** -24).all()


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [20, 200])
def test_states(svx, rows, d, ty):
    """An item to each SM, all of the same states (KV heads broadcast), and so one segment of all of them; the last of three lengths hides
    a part of a tile, and scores grow over the keys, so that the reference moves between the sums."""
    t, states = TYPES[ty], 1 << 21
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(rows)
    k = 0.5 * torch.randn((states, d), generator=g, device="cuda")
    k[:, 0] = torch.linspace(-4, 4, states, device="cuda")
    k, v = k.to(t), torch.rand((states, d), generator=g, device="cuda").to(t)
    q = (0.5 * torch.randn((1, sms, rows, d), generator=g, device="cuda"))
    q[..., 0] = d ** 0.5 / 2  # scores rise by 4 on the way
    q = q.to(t)
    ks, vs = (x.view(1, states, 1, d).expand(1, states, sms, d) for x in (k, v))
    o, lse = torch.full_like(q, 7.0), torch.zeros((1, sms, rows), device="cuda")
    for n in (states, 40000, 3 * (1 << 19) + 77):
        svx.cross_attn(q, ks, vs, o, lse, lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        for h in (0, sms - 1):
            want = attend64(q[0, h], k[:n], v[:n], d ** -0.5)
            near(o[0, h], lse[0, h], want, torch.finfo(t).eps / 2 if rows > 128 else 2.0 ** -15, -(-n // 128))


@pytest.mark.parametrize("batch", [12, 100])
def test_a_shared_prefix(svx, batch):
    """3 million slots of each of 16 KV heads (in 24 pages that the table names over and over), cut over the CTAs, so that segments begin and
    end within items, and slots of the requests' own behind them."""
    d, heads, page, t = 64, 16, 8192, torch.float16
    g = torch.Generator(device="cuda").manual_seed(batch)
    k = torch.randn((25, page, heads, d), generator=g, device="cuda").to(t)
    v = torch.rand((25, page, heads, d), generator=g, device="cuda").to(t)
    c = svx.PagedCache(k, v)
    q = torch.randn((batch, 2 * heads, 1, d), generator=g, device="cuda").to(t)
    order = torch.randint(0, 24, (1, 384), generator=g, device="cuda", dtype=torch.int32)
    n = 384 * page - 1000
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens = torch.full((batch, 1), 24, dtype=torch.int32, device="cuda"), torch.arange(batch, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.zeros((batch, 2 * heads, 1), device="cuda")
    c.decode_shared(q, order, ints(n), ints(0, batch), table, lens, o, lse, max_len=batch)
    assert not c.check()
    for h in (0, 7, 15):
        far = [x[order[0].long(), :, h].reshape(-1, d)[:n] for x in (k, v)]
        for b in (0, batch // 2, batch - 1):
            x = slice(2 * h, 2 * h + 2)
            want = attend64(q[b, x, 0], *(torch.cat((y, z[24, :b, h])) for y, z in zip(far, (k, v))), d ** -0.5)
            near(o[b, x, 0], lse[b, x, 0], want, 2.0 ** -11 if 2 * batch > 128 else 2.0 ** -15, -(-n // 128))
