"""The residual stream: rows of a few lanes, of one piece to a thread and of three, in numbers that leave warps and blocks partly
empty and make them take several turns.  Inputs, definition and bounds: test_gpu_residual."""
import pytest
import torch

from test_gpu_residual import cuda, inputs, near, reference, svx  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", ["fp16", "fp32"])
@pytest.mark.parametrize("rows, dim", [(1, 64), (2, 8), (3, 56), (5, 128), (6, 72), (17, 64), (1001, 120), (60001, 64), (30003, 72), (5003, 136),
                                       (700, 520), (1300, 648), (1217, 768), (305, 8200), (153, 12288), (304, 12296)])
def test_rows_of_any_width(svx, rows, dim, stream):  # noqa: F811
    s = inputs(rows, dim, "fp16", stream, "weights", "element" if rows % 2 else "channel", seed=rows)
    z, e, x, ex = reference(s, True, "sigmoid", 0.9, 1.1)
    c = cuda(s)
    # rows apart in wider buffers: what lies between them and behind the last one stays
    ho = torch.full((rows + 3, dim + 8), 7.0, dtype=c["h"].dtype, device="cuda")
    xo = torch.full((rows + 3, dim + 24), 7.0, dtype=c["y"].dtype, device="cuda")
    svx.residual_norm(c["h"], c["y"], ho[:rows, :dim], xo[:rows, :dim], norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5,
                      gate=c["gate"], act="sigmoid", alpha=0.9, beta=1.1)
    near(ho[:rows, :dim], z, e)
    near(xo[:rows, :dim], x, ex)
    assert (ho[rows:] == 7).all() and (ho[:, dim:] == 7).all() and (xo[rows:] == 7).all() and (xo[:, dim:] == 7).all()
    svx.residual_norm(c["h"], c["y"], c["h"], c["y"], norm=c["norm"], post_norm=c["post_norm"], post_eps=1e-5, gate=c["gate"],
                      act="sigmoid", alpha=0.9, beta=1.1)  # in place
    assert torch.equal(c["h"], ho[:rows, :dim]) and torch.equal(c["y"], xo[:rows, :dim])
