"""The Python side of the 8-bit cache calls without a GPU."""
import contextlib

import pytest
import torch

from gist_token_chunk_b200 import ssa


class FakeCuda:
    """Two devices: which one is current when the library is called."""

    def __init__(self, monkeypatch):
        self.now, self.seen = 0, []
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.now)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(ssa, "_stream", lambda s: ("current", self.now) if s is None else s)
        monkeypatch.setattr(ssa.lib, "ssa_cache_get_status", self.status)

    @contextlib.contextmanager
    def device(self, d):
        was = self.now
        self.now = was if d is None else torch.device(d).index
        yield
        self.now = was

    def status(self, code, stream):
        self.seen.append((self.now, stream))
        code._obj.value = ssa.SSA_ERR_DEVICE_STATUS if self.now == 1 else 0
        return ssa.SSA_OK


def test_status_of_another_device(monkeypatch):
    """The status word is the asked device's, read with that device and its stream current."""
    cuda = FakeCuda(monkeypatch)
    assert ssa.ssa_cache_get_status() == 0
    assert cuda.seen.pop() == (0, ("current", 0))
    for d in (1, "cuda:1", torch.device("cuda", 1)):
        assert ssa.ssa_cache_get_status(device=d) == ssa.SSA_ERR_DEVICE_STATUS
        assert cuda.seen.pop() == (1, ("current", 1))
    assert ssa.ssa_cache_get_status(device="cuda") == 0 and cuda.now == 0
    assert ssa.ssa_cache_get_status(stream=7, device=1) == ssa.SSA_ERR_DEVICE_STATUS
    assert cuda.seen.pop() == (1, 7)
    with pytest.raises(ValueError):
        ssa.ssa_cache_get_status(device="cpu")


def test_status_takes_the_streams_device(monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 99

    cuda = FakeCuda(monkeypatch)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    s = Stream()
    assert ssa.ssa_cache_get_status(s) == ssa.SSA_ERR_DEVICE_STATUS
    assert cuda.seen.pop() == (1, s)
    assert ssa.ssa_cache_get_status(s, device=1) == ssa.SSA_ERR_DEVICE_STATUS
    with pytest.raises(ValueError):
        ssa.ssa_cache_get_status(s, device=0)
