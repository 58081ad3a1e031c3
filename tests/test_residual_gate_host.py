"""residual_norm with an activation and an optional gate, without a GPU: what reaches the native call."""
import pytest


@pytest.fixture()
def calls(monkeypatch):
    from speculative_decoding_verification_chunked_gb300 import svx

    class Native:
        def residual_norm(self, *args):
            self.args = args

    native = Native()
    monkeypatch.setattr(svx, "_native_module", native)
    return svx, native


@pytest.mark.parametrize("act", [None, "tanh", "sigmoid"])
def test_an_activation_has_nothing_to_work_on_without_a_gate(calls, act):
    svx, native = calls
    svx.residual_norm("h", "y", "h_out", "x_out", gate=None, act=act)
    without = native.args
    svx.residual_norm("h", "y", "h_out", "x_out")
    assert without == native.args and without[8] is None and without[9] == 0


def test_an_activation_goes_with_its_gate(calls):
    svx, native = calls
    svx.residual_norm("h", "y", "h_out", "x_out", gate="gate", act="tanh")
    assert native.args[8:10] == ("gate", 1)
    svx.residual_norm("h", "y", "h_out", "x_out", act="sigmoid")  # no gate is passed: the native call refuses it
    assert native.args[8:10] == (None, 2)


@pytest.mark.parametrize("kw", [dict(gate=None), dict(gate="gate"), dict()], ids=str)
def test_an_unknown_activation_is_refused_all_the_same(calls, kw):
    svx, _ = calls
    with pytest.raises(svx.SvxError) as e:
        svx.residual_norm("h", "y", "h_out", "x_out", act="relu", **kw)
    assert e.value.status == svx.ERR_INVALID_ARG
