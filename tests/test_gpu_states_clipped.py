"""Whole tiles, which come in by tensor map, described as lying past the end of k and v: the bounds-checked library reports it, reads nothing
there and leaves the other requests alone; the other library takes no notice."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.environ.get("SVX_LIBRARY") == "checked"


@pytest.fixture(scope="module")
def svx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_chunked_gb300 import svx as mod
    return mod


def clip(svx, n):
    assert svx.lib.svx_debug_clip_paged(2, n) == svx.OK


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("masked", [False, True])
def test_states(svx, n, masked):
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((3, 2, n, 64), (3, 512, 1, 64), (3, 512, 1, 64)))
    mask = torch.rand((3, 512), generator=g, device="cuda") < 0.9 if masked else None
    want, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    svx.cross_attn(q, k, v, want, mask=mask, status=status)
    assert status.item() == 0
    for end in (64 * (2 * 512 + 200), 64 * (2 * 512 + 128), 64 * (3 * 512 - 1)):  # within the third request's states
        o = torch.zeros_like(q)
        try:
            clip(svx, end)
            svx.cross_attn(q, k, v, o, mask=mask, status=status)
        finally:
            clip(svx, -1)
        assert (status.item() != 0) == CHECKED
        assert torch.equal(o[:2], want[:2]) and torch.equal(o[2], want[2]) != CHECKED
        status.zero_()


@pytest.mark.parametrize("batch", [40, 200])
@pytest.mark.parametrize("page", [8, 64, 128])
def test_prefixes(svx, page, batch):
    g = torch.Generator(device="cuda").manual_seed(page)
    pages = 1024 // page
    k, v = (torch.randn((pages + 1, page, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    c = svx.PagedCache(k, v)
    q = torch.randn((batch, 1, 1, 64), generator=g, device="cuda").bfloat16()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    far, table, lens = torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.zeros((batch, 1), dtype=torch.int32, device="cuda"), ints(*[0] * batch)

    def run():
        o, lse = torch.zeros_like(q), torch.zeros((batch, 1, 1), device="cuda")
        c.decode_shared(q, far, ints(1024), ints(0, batch), table, lens, o, lse)
        return o

    want = run()
    assert not c.check()
    for end in (64 * 1000, 64 * 512, 64 * 1023):
        try:
            clip(svx, end)
            o = run()
        finally:
            clip(svx, -1)
        assert c.check() == CHECKED and torch.equal(o, want) != CHECKED


@pytest.mark.skipif(CHECKED, reason="this is the run on the bounds-checked library")
def test_on_the_bounds_checked_library(svx):
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_states_clipped.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, SVX_LIBRARY="checked"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
