"""The build itself: the libraries of the C ABI depend on neither PyTorch nor the binding's compiler call."""
import os
import sys

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module on one small translation unit, with its outputs elsewhere."""
    from speculative_decoding_verification_chunked_gb300 import build as b
    try:
        b.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    monkeypatch.setattr(b, "SOURCES", ["svx_width.cu"])
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    for name in ("LIB", "LIB_CHECKED", "LIB_TORCH"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    return b


@pytest.mark.parametrize("torch", ["none", "without CUDA"])
def test_the_libraries_build_without_pytorch(build, monkeypatch, capsys, torch):
    if torch == "none":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    else:
        monkeypatch.setattr(pytest.importorskip("torch").version, "cuda", None)
    open(build.LIB_TORCH, "w").close()  # of an earlier build
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.LIB_CHECKED) and not os.path.exists(build.LIB_TORCH)
    assert "svx_torch.so is not built" in capsys.readouterr().err


@pytest.mark.parametrize("command", [[sys.executable, "-c", "raise SystemExit('no headers')"], ["/nonexistent/g++"]], ids=["fails", "missing"])
def test_a_failure_of_the_binding_is_raised_and_leaves_the_libraries(build, monkeypatch, command):
    monkeypatch.setattr(build, "torch_command", lambda out: command)
    with pytest.raises(RuntimeError, match="svx_torch.so is not"):
        build.build(checked=False)
    assert os.path.exists(build.LIB) and not os.path.exists(build.LIB_TORCH)


def test_the_binding_is_built_where_pytorch_is(build):
    pytest.importorskip("torch")
    build.build(checked=False)
    assert os.path.exists(build.LIB) and os.path.exists(build.LIB_TORCH)
