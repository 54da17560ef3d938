"""CPU checks of the frame-aware operators' binding: on which stream and device a call runs."""

from __future__ import annotations

from types import SimpleNamespace

import pytest

from fixed_pattern_sparse_b200 import frames


def test_a_stream_of_another_device_is_refused():
    """The kernels would run on the stream's device and read the tensors' memory of the other one."""
    ran = []
    with pytest.raises(ValueError, match="cuda:1"):
        frames._on(1, SimpleNamespace(device_index=0, cuda_stream=0), ran.append)
    assert not ran


def test_a_stream_of_the_tensors_device_is_used(monkeypatch):
    """Current for the call, with the tensors' device, whichever device is current outside."""
    entered = []

    class Guard:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            entered.append(self.what)

        def __exit__(self, *_):
            entered.append(None)

    monkeypatch.setattr(frames.torch.cuda, "device", Guard)
    monkeypatch.setattr(frames.torch.cuda, "stream", Guard)
    stream = SimpleNamespace(device_index=1, cuda_stream=77)
    assert frames._on(1, stream, lambda st: (st, list(entered))) == (77, [1, stream])
    assert entered == [1, stream, None, None]
