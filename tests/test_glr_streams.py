"""Which stream a glr_scan or ckpt8 call takes for its `stream` argument, with
torch's CUDA streams replaced by stand-ins: no GPU is needed."""
import contextlib

import pytest
import torch


class Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", device)


@pytest.fixture
def on(monkeypatch):
    """_on with stand-ins; the stream whose context it entered is the last of `entered`."""
    import delta_rule_memory_gb300 as sdm
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: Stream(("pool", h) if h == 0 else h, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d: Stream(0, d))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: entered[-1])
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return sdm._on, entered


@pytest.mark.parametrize("stream", [0, 1, type("Raw", (), {"cuda_stream": 0})()], ids=["null", "legacy", "object"])
def test_the_default_stream_s_handles(on, stream):
    call, entered = on
    with call(0, stream) as handle:
        assert handle == 0
    assert len(entered) == 1


def test_other_streams(on):
    call, entered = on
    with call(0, 4096) as handle:
        assert handle == 4096
    mine = Stream(8192)
    with call(0, mine) as handle:
        assert handle == 8192
    assert entered[-1] is mine


def test_a_stream_of_another_device_is_refused(on):
    """The kernel would run there, on this device's addresses."""
    call, entered = on
    with pytest.raises(ValueError, match="cuda:0"):
        call(0, Stream(4096, device=1))
    with pytest.raises(ValueError, match="cuda:1"):
        call(1, Stream(4096))
    assert not entered
