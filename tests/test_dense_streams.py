"""Which stream the dense-state layer's calls run on, without a GPU: what the `stream` argument
stands for, with torch's stream types replaced by ones that need no device."""

import contextlib

import pytest
import torch

from sparse_memory_linear_b200 import _binding as b


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device = handle, device


class External(Stream):
    def __init__(self, handle, device=None):
        assert handle != 0, "a null handle gives a stream of the pool"
        super().__init__(handle, device)


@pytest.fixture
def used(monkeypatch):
    """The streams that were made the current one, in order."""
    entered = []

    @contextlib.contextmanager
    def current(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0, device))
    monkeypatch.setattr(torch.cuda, "stream", current)
    return entered


DEV = torch.device("cuda", 1)


def test_null_handle_is_the_default_stream(used):
    """0 is what torch.cuda.default_stream().cuda_stream gives."""
    with b._scope(0, DEV):
        pass
    assert used[0].cuda_stream == 0 and used[0].device == DEV


def test_handles_and_streams_are_used_as_given(used):
    own = Stream(77, DEV)
    with b._scope(own, DEV), b._scope(1234, DEV):
        pass
    assert used[0] is own
    assert used[1].cuda_stream == 1234 and used[1].device == DEV


def test_streams_of_another_device_are_refused(used):
    """The call would run on the current stream of its tensors' device, not on the given one."""
    with pytest.raises(ValueError):
        b._scope(Stream(77, torch.device("cuda", 0)), DEV)
    assert not used
