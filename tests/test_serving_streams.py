"""The stream that a serving call is given is the one that it runs on (host side; no GPU)."""
import contextlib
import types

import pytest
import torch


@pytest.fixture()
def calls(monkeypatch):
    """What would be made current, by fakes of torch's streams."""
    made = []

    class Stream:
        def __init__(self, device, cuda_stream):
            self.device, self.cuda_stream = torch.device(device), cuda_stream

    class ExternalStream(Stream):
        def __init__(self, handle, device=None):
            assert handle != 0, "torch takes a pointer of 0 for none given"
            super().__init__(device, handle)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ExternalStream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(device, 0))

    def stream(s):
        made.append((s.device, s.cuda_stream))
        return contextlib.nullcontext()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    return types.SimpleNamespace(made=made, Stream=Stream)


def _made(calls, stream, device):
    from hashed_gram_memory_amd import serving
    with serving._on(stream, types.SimpleNamespace(device=torch.device(device))):
        pass
    return calls.made[-1]


@pytest.mark.parametrize("device", ["cuda:0", "cuda:1"])
def test_handles(calls, device):
    for handle in (0, 0x55D0):
        assert _made(calls, handle, device) == (torch.device(device), handle)


def test_streams_of_the_device_alone(calls):
    assert _made(calls, calls.Stream("cuda:1", 0x77), "cuda:1") == (torch.device("cuda:1"), 0x77)
    with pytest.raises(ValueError):
        _made(calls, calls.Stream("cuda:0", 0x77), "cuda:1")


def test_host_tensors_are_refused_with_a_stream_too():
    import hashed_gram_memory_amd as hg
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    cache = torch.zeros((2, 8, 16, 64), dtype=torch.bfloat16)
    for call in (lambda: hg.qk_norm_rope(q, None, stream=0),
                 lambda: hg.kv_append(q, q, cache, cache, torch.zeros(1, dtype=torch.int64), stream=7),
                 lambda: hg.paged_attention(q, cache, cache, torch.zeros((1, 2), dtype=torch.int32),
                                            torch.ones(1, dtype=torch.int32), stream=0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        hg.kv_append([1], q, cache, cache, torch.zeros(1, dtype=torch.int64), stream=0)
