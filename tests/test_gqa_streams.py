"""Streams of the grouped-head calls, host side: which device and stream a call moves to."""
import contextlib

import pytest
import torch

import long_context_sparse_10_b200 as csa


class FakeStream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def cuda(monkeypatch):
    entered = []

    @contextlib.contextmanager
    def enter(x):
        entered.append(x)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: FakeStream(device.index))
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "device", enter)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return entered


def test_a_stream_of_another_device_is_refused(cuda):
    with pytest.raises(ValueError, match="stream is on cuda:1, not on cuda:0"):
        csa._elsewhere(torch.device("cuda", 0), FakeStream(1))
    with pytest.raises(ValueError, match="stream is on cuda:0, not on cuda:2"):
        csa._elsewhere(torch.device("cuda", 2), FakeStream(0))
    assert cuda == []


def test_a_stream_of_the_tensors_device_becomes_the_current_one(cuda):
    st = FakeStream(1)
    with csa._elsewhere(torch.device("cuda", 1), st):
        assert cuda == [st]
    with csa._elsewhere(torch.device("cuda", 1), 4096):
        assert cuda[1].device == torch.device("cuda", 1)


def test_no_stream(cuda):
    assert csa._elsewhere(torch.device("cuda", 0), None) is None
    with csa._elsewhere(torch.device("cuda", 3), None):
        assert cuda == [torch.device("cuda", 3)]
    with pytest.raises(ValueError, match="CUDA"):
        csa._elsewhere(torch.device("cpu"), None)
