"""Which stream the binding takes when it is given none, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
E = pytest.importorskip("hashed_gram_conditional_amd")

from hashed_gram_conditional_amd import _binding  # noqa: E402


class _Stream:
    cuda_stream = 0x51


@pytest.fixture
def initialised(monkeypatch):
    """torch with a current device 1 whose current stream is 0x51."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream)


def test_the_handle_of_the_current_device_s_stream(initialised, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x70 + device, raising=False)
    assert _binding._stream(None) == 0x71


def test_the_public_way_without_the_handle_s_function(initialised, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert _binding._stream(None) == 0x51


def test_a_given_stream_is_taken_as_it_is():
    assert _binding._stream(0) == 0 and _binding._stream(0x99) == 0x99
    assert _binding._stream(_Stream) == 0x51
