"""The tests of attention to an encoder's states, behind shared prefixes and of the residual stream again on the bounds-checked library
(libsvx_checked.so): every row of K and V that the kernels read is checked against its buffer."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_states_suite_on_the_bounds_checked_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, SVX_LIBRARY="checked")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_cross.py",
           "tests/test_gpu_shared.py", "tests/test_gpu_residual.py", "tests/test_gpu_states_edges.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
