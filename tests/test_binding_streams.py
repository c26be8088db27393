"""The stream that the long-context operators' binding launches on, without a GPU: torch's device and stream functions are
stood in for."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def cuda(monkeypatch):
    """binding._cuda on device 1 of a process whose current stream there is number 7."""
    from decoder_only_transformer_gpt_gb300 import binding
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 7, raising=False)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    binding._cuda_up = False                                             # asks torch again, here and after the test
    yield binding._cuda
    binding._cuda_up = False


def test_the_current_stream(cuda):
    assert cuda(None)[1:] == (1, 7)


def test_a_stream_of_the_current_device(cuda):
    assert cuda(types.SimpleNamespace(cuda_stream=9, device_index=1))[1:] == (1, 9)


def test_a_stream_of_another_device_is_refused(cuda):
    with pytest.raises(ValueError, match="stream: of device 0"):
        cuda(types.SimpleNamespace(cuda_stream=9, device_index=0))


def test_a_torch_without_the_short_names(cuda, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getDevice")
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=11))
    assert cuda(None)[1:] == (1, 11)
