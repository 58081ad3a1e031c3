"""Edges of the paged-cache operators on the GPU: calls that the header allows and whose results hang on one detail.

Bounds are derived at each test; u = torch.finfo(type).eps / 2 is a rounding to the output type.
"""
import math

import numpy as np
import pytest
import torch

from paged_reference import heads64

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ heads


def pair_terms(y, pos, inv_freq, neighbours):
    """|y_a cos t| + |y_b sin t| and |y_b cos t| + |y_a sin t| at their places: the size that a rotated value's error goes by."""
    half = len(inv_freq)
    ang = torch.as_tensor(pos, dtype=torch.float64)[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(ang).abs()[:, None], torch.sin(ang).abs()[:, None]
    out = y.abs().clone()
    ia = torch.arange(half) * 2 if neighbours else torch.arange(half)
    ib = ia + (1 if neighbours else half)
    a, b = y[..., ia].abs(), y[..., ib].abs()
    out[..., ia], out[..., ib] = a * c + b * s, b * c + a * s
    return out


@pytest.mark.parametrize("zero", ["first", "second", "none"])
@pytest.mark.parametrize("neighbours", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("d,ty", [(128, "bf16"), (128, "fp16"), (64, "fp16"), (64, "bf16")])
def test_small_angles_keep_their_sine(svx, d, ty, neighbours, zero):
    """A pair with one member zero shows sine and cosine themselves, down to angles of 1e-7: each output is within its own rounding.
    In fp32 (u' = 2^-24): angle, sine and cosine within 4 u' relative, two products and a sum 2 u', the scale 1 u': under 2^-20 of
    |y_a cos t| + |y_b sin t|, and a sum rounded to the type.  (The angle's phase is off by 2^-55 |pos| turns at most: nothing beside.)"""
    t, n = TYPES[ty], 600
    g = torch.Generator().manual_seed(21)
    x = torch.randn((1, n, 2, d), generator=g).to(t)
    first = torch.zeros(d, dtype=torch.bool)
    if neighbours:
        first[0::2] = True
    else:
        first[:d // 2] = True
    if zero != "none":
        x[..., first if zero == "first" else ~first] = 0
    pos = torch.cat([torch.arange(-100, 300), torch.randint(-2 ** 20, 2 ** 20, (n - 400,), generator=g)]).to(torch.int32)[None]
    inv = [1e6 ** (-2.0 * i / d) for i in range(d // 2)]
    inv[1], inv[3] = 3e-7, 1.0 / 65536  # (positions times 2^-16 reach the quadrants' borders to within an ulp)
    inv[5] = math.pi / 4
    qo, ko = torch.empty((1, 1, n, d), dtype=t, device="cuda"), torch.empty((1, n, 1, d), dtype=t, device="cuda")
    xc = x.cuda()
    svx.qk_norm_rope(xc[:, :, :1], xc[:, :, 1:], None, pos.cuda(), svx.Rope(d, inv_freq=inv, neighbours=neighbours), qo, ko, eps=None)
    for got, h in ((qo[0].transpose(0, 1), 0), (ko[0], 1)):
        z, _ = heads64(x[0, :, h:h + 1], None, None, pos[0], inv, neighbours)
        size = pair_terms(x[0, :, h:h + 1].double(), pos[0], inv, neighbours)
        # the reference's own angle: 64-bit products of up to 2^20 are off by 2^-33 radians at most
        bound = z.abs() * torch.finfo(t).eps / 2 + size * 2.0 ** -20 + x[0, :, h:h + 1].double().abs().amax() * 2.0 ** -33 \
            + torch.finfo(t).tiny * torch.finfo(t).eps
        err = (got.double().cpu() - z).abs()
        assert (err <= bound).all(), f"{float((err / bound).max()):.2f} times the bound at {int((err > bound).sum())} elements"


# ------------------------------------------------------------------ one-token attention


@pytest.mark.parametrize("which", ["k", "v"])
def test_decode_refuses_a_workspace_in_the_pools(svx, which):
    """The workspace's size needs the device's SM count, so this is seen here: a workspace that begins in a pool, ends in it, or lies
    beside it."""
    n = 4 * 16 * 2 * 64
    need = svx.ctypes.c_int64(0)
    arena = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    mine = arena[1 << 23:(1 << 23) + 2 * n].view(torch.bfloat16).view(4, 16, 2, 64)
    other = torch.zeros_like(mine)
    cache = svx.PagedCache(*((mine, other) if which == "k" else (other, mine)))
    q, o = (torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, table, lens = torch.zeros((1, 4, 1), device="cuda"), i32([[0, 1, 2]]), i32([40])
    p = svx.Pages.from_buffer_copy(cache._pages)
    p.table, p.max_pages = table.data_ptr(), 3
    assert svx.lib.svx_paged_decode_workspace(svx.ctypes.byref(p), 1, 4, 0, 0, svx.ctypes.byref(need)) == svx.OK
    size = (need.value + 255) // 256 * 256
    for at in ((1 << 23), (1 << 23) + 2 * n - 256, (1 << 23) - size + 256):
        with pytest.raises(svx.SvxError, match="overlap"):
            cache.decode(q, table, lens, o, lse, workspace=arena[at:at + size])
    for at in ((1 << 23) + 2 * n, (1 << 23) - size):
        cache.decode(q, table, lens, o, lse, workspace=arena[at:at + size])
    assert not cache.check()


# ------------------------------------------------------------------ the bounds-checked library


def test_strays_name_the_buffer_that_they_left(svx):
    """With buffers described as smaller than they are (svx_debug_clip_paged), the checked library skips what lies past the end and names the
    buffer; the other library, and the next call, do all of it."""
    checked = "bounds-checked" in svx.version()
    g = torch.Generator().manual_seed(22)
    n, hq, hkv, d, page, t = 6, 4, 2, 64, 4, torch.bfloat16
    x = torch.randn((1, n, hq + 2 * hkv, d), generator=g).to(t).cuda()
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    pos, rope, table, start = i32([list(range(n))]), svx.Rope(d), i32([[0, 1]]), i32([1])
    qo = torch.zeros((1, hq, n, d), dtype=t, device="cuda")
    ko, vo = (torch.zeros((1, n, hkv, d), dtype=t, device="cuda") for _ in range(2))
    kp, vp = (torch.zeros((2, page, hkv, d), dtype=t, device="cuda") for _ in range(2))
    cache, status = svx.PagedCache(kp, vp), i32([0])
    o, lse, lens = torch.zeros((1, hq, 1, d), dtype=t, device="cuda"), torch.zeros((1, hq, 1), device="cuda"), i32([n + 1])
    acc = torch.zeros((1, hkv, 2 * page), device="cuda")
    spos = torch.zeros((1, hkv, 2 * page), dtype=torch.int32, device="cuda")

    def dense():
        svx.qk_norm_rope(q, k, v, pos, rope, qo, ko, vo, status=status)
        return status

    def append():
        cache.append(q, k, v, pos, rope, table, start, qo)
        return cache.status

    def decode():
        cache.decode(q[:, :1].transpose(1, 2).contiguous(), table, lens, o, lse)
        return cache.status

    def evict():
        cache.evict(table, lens, 3, 0, 3, i32([8]), acc, spos.copy_(torch.arange(2 * page, device="cuda").int().expand_as(spos)), acc,
                    spos, i32([0]))
        return cache.status

    def clip(buffer, elements):
        assert svx.lib.svx_debug_clip_paged(buffer, elements) == svx.OK
    inside, outside, pool = 1 << 17, 1 << 18, 1 << 19
    cases = [(dense, 0, 3 * (hq + 2 * hkv) * d, inside), (append, 0, 3 * (hq + 2 * hkv) * d, inside), (dense, 1, 2 * hkv * d, outside),
             (append, 1, 2 * hkv * d, outside), (append, 2, page * hkv * d, pool), (decode, 2, page * hkv * d, pool), (evict, 2, page * hkv * d, pool)]
    for call, buffer, elements, bit in cases:
        word = call()
        assert int(word) == 0, call.__name__
        for y in (qo, ko, vo):
            y.zero_()
        try:
            clip(buffer, elements)
            call()
        finally:
            clip(buffer, -1)
        assert int(word) == (4 | bit if checked else 0), (call.__name__, buffer, hex(int(word)))
        word.zero_()
        if checked and buffer == 1:
            assert (qo.view(-1)[2 * hkv * d:] == 0).all() and (qo.view(-1)[:2 * hkv * d] != 0).any()
            if call is dense:
                assert (ko.view(-1)[2 * hkv * d:] == 0).all() and (vo.view(-1)[2 * hkv * d:] == 0).all() and (vo.view(-1)[:2 * hkv * d] != 0).any()
        call()
        assert int(word) == 0
    assert svx.lib.svx_debug_clip_paged(3, 0) == svx.ERR_INVALID_ARG
