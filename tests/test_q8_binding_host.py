"""The Python side of the rotary and 8-bit cache calls without a GPU."""
import contextlib
import math
import os
import subprocess
import sys

import pytest
import torch

from gist_token_chunk_b200 import build, ssa


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


WITHOUT = """
from gist_token_chunk_b200 import build
build.binding_path = lambda: build.LIB + ".none"
import torch
from gist_token_chunk_b200 import ssa
shape = ssa.make_shape(2, 8, 2, 64, 1024, ssa.SSA_BF16)
assert ssa.ssa_workspace_size(shape, 64, 8, 4) > 0
assert ssa.ssa_rope_freqs(64)[0].shape == (32,)
try:
    ssa.ssa_rope(torch.zeros(1, 1, 1, 64), None, torch.zeros(1), torch.zeros(32))
except ImportError as e:
    print("raised" if "build.py" in str(e) else e)
"""


def test_the_library_without_its_binding():
    """A binding that does not load takes its own calls with it and no others."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "raised", r.stderr[-2000:]


def test_the_binding_is_built_for_its_torch(monkeypatch):
    """Up to date for this Python and torch; another torch has it compiled anew."""
    started = []
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd: started.append(cmd))
    assert build._start_binding(False) is None and not started
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert build.binding_path() != here
    _, out = build._start_binding(False)
    assert started and out.startswith(build.binding_path())


@pytest.mark.parametrize("length", [65536.0, 131072.0, 1e6, 1e9])
def test_ramped_frequencies_of_a_long_original_length(length):
    """A last pair that makes more than `low` turns is not slowed as if it made fewer: the ramp
    ends past it, and no frequency falls when the original length grows."""
    low, high, factor, r, base = 1.0, 32.0, 16.0, 64, 10000.0
    f0, _ = ssa.ssa_rope_freqs(r, base)
    f, _ = ssa.ssa_rope_freqs(r, base, ssa.SSA_ROPE_RAMPED, factor, low, high, length)
    turns = length * f0 / (2 * math.pi)
    first, last = (r * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low))
    first, last = max(math.floor(first), 0), min(math.ceil(last), r - 1)
    assert float(turns[-1]) > low and last > r // 2 - 1
    for i, (a, b) in enumerate(zip(f0.tolist(), f.tolist())):
        w = min(max((i - first) / (last - first), 0.0), 1.0)
        assert b == pytest.approx((1 - w) * a + w * a / factor, rel=1e-13)
    shorter, _ = ssa.ssa_rope_freqs(r, base, ssa.SSA_ROPE_RAMPED, factor, low, high, length * 0.9)
    assert (f >= shorter).all()
