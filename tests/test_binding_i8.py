"""Buffers of another device than the current one are refused by the 8-bit operators and the
gradients when no stream is given, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
E = pytest.importorskip("hashed_gram_conditional_amd")

from tests.test_binding_stream import _Tensor, initialised  # noqa: E402,F401


def _calls(t, stream=None):
    """Every call of the four with nothing to do."""
    d = E.forward_desc(1, 0, 1, 64, 0, E.ROW_E4M3_E8M0_264, 256)
    saved = E.gate_saved(t, E.I8, t, t, E.I8, t)
    return [lambda: E.engram_quantize_i8(t, E.F32, 0, 64, 0, 64, E.SCALE_F32, t, t, t, stream),
            lambda: E.engram_project_i8(t, t, t, t, t, E.BF16, 0, 64, 64, None, 0, stream),
            lambda: E.engram_gate_grad(d, t, 10, saved, t, t, t, t, t, None, None, 1, None, 0, stream),
            lambda: E.engram_project_grad(t, t, t, t, E.F32, 1, 0, 64, 64, None, 0, stream)]


@pytest.mark.parametrize("k", range(4))
def test_buffers_of_another_device_are_refused(initialised, k):      # noqa: F811
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        _calls(_Tensor(0))[k]()
    _calls(_Tensor(1))[k]()
    _calls(_Tensor(0), 0x99)[k]()        # a stream of their device given
