"""Which stream the binding takes when it is given none, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
E = pytest.importorskip("hashed_gram_conditional_amd")

from hashed_gram_conditional_amd import _binding  # noqa: E402


class _Stream:
    cuda_stream = 0x51


@pytest.fixture
def initialised(monkeypatch):
    """torch with a current device 1 whose current stream is 0x51 (its handle 0x71 where the
    handle's own function is asked)."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x70 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream)


def test_the_handle_of_the_current_device_s_stream(initialised):
    assert _binding._stream(None) == 0x71


@pytest.mark.parametrize("name", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_public_way_without_the_handle_s_function(initialised, monkeypatch, name):
    monkeypatch.delattr(torch._C, name, raising=False)
    assert _binding._stream(None) == 0x51


def test_a_given_stream_is_taken_as_it_is():
    assert _binding._stream(0) == 0 and _binding._stream(0x99) == 0x99
    assert _binding._stream(_Stream) == 0x51


class _Tensor:
    """A device tensor of which the host code only asks what it needs to know."""
    is_cuda = True

    def __init__(self, device):
        self.device_index = device

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def is_pinned(self):
        return False

    def data_ptr(self):
        return 0x10000


def _calls(t, stream=None):
    """Every call of the lookup, its gradient, the quantiser and the product with nothing to do."""
    d = E.embed_desc(0, 0, 16)
    return [lambda: E.engram_embed(d, t, t, t, stream),
            lambda: E.engram_embed_grad_dense(d, t, t, t, 1, t, 1 << 40, stream),
            lambda: E.engram_quantize_mx4(t, E.F32, 0, 64, 0, 64, t, t, t, stream),
            lambda: E.engram_project_mx4(t, t, E.MX_E2M1, t, t, t, 0, 256, 64, None, 0, stream)]


@pytest.mark.parametrize("k", range(4))
def test_buffers_of_another_device_are_refused(initialised, k):
    _calls(_Tensor(1))[k]()
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        _calls(_Tensor(0))[k]()
    _calls(_Tensor(0), 0x99)[k]()        # a stream of their device given


def test_the_sparse_gradient_refuses_them_too(initialised):
    t, d = _Tensor(0), E.embed_desc(0, 0, 16)
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        E.engram_embed_grad(d, t, t, t, t, t, t, 0)
