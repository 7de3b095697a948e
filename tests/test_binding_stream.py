"""The stream that a call without one is given: torch's current stream of the
current device, found through torch's public interface where the short way to
its handle is missing (no GPU: the interface is replaced)."""
import types

import pytest
import torch

import combine_ep_plan_amd as ep


class Stream:
    cuda_stream = 77


@pytest.fixture
def fake(monkeypatch):
    calls = []
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: calls.append("init"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: calls.append("current_stream") or Stream())
    return calls


def test_without_the_short_way_the_public_one_is_taken(monkeypatch, fake):
    for missing in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        bare = types.SimpleNamespace(**{n: (lambda *a: 5) for n in
                                        ("_cuda_getCurrentRawStream", "_cuda_getDevice") if n != missing})
        assert ep._stream_finder(bare)() == 77, missing
    assert fake == ["current_stream"] * 2


def test_the_short_way_asks_for_the_current_device(monkeypatch, fake):
    asked = []
    short = types.SimpleNamespace(_cuda_getDevice=lambda: 3,
                                  _cuda_getCurrentRawStream=lambda d: asked.append(d) or 41)
    assert ep._stream_finder(short)() == 41 and asked == [3] and fake == []


def test_the_device_is_looked_up_once_torch_is_initialised(monkeypatch, fake):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    short = types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda d: 9)
    assert ep._stream_finder(short)() == 9 and fake == ["init"]


def test_given_streams_pass_through():
    assert ep._stream(0) == 0 and ep._stream(12) == 12 and ep._stream(Stream()) == 77
