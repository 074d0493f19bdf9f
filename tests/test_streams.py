"""Buffers that the binding allocates for a call on another stream than the current one: whose
memory they come from, and who is told of them.  On the CPU, with stand-ins for streams."""
import contextlib

import pytest

import nvfp4_w4a4_quantized_02_b200 as nv


class _Stream:
    def __init__(self, raw, device=0):
        self.cuda_stream = raw
        self.device = type("D", (), {"index": device})


class _Buffer:
    def __init__(self, pool):
        self.pool, self.told = pool, []

    def record_stream(self, s):
        self.told.append(s)


@pytest.fixture
def world(monkeypatch):
    import torch
    now = [_Stream(7)]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()
    monkeypatch.setattr(nv, "_raw_stream", lambda dev: now[-1].cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    return lambda: _Buffer(now[-1].cuda_stream)


def test_current_stream_needs_nothing(world):
    for stream in (None, _Stream(7)):
        t = nv._made(0, stream, world)
        assert t.pool == 7 and not t.told


def test_another_stream_gives_the_memory_and_the_current_one_is_told(world):
    t = nv._made(0, _Stream(9), world)
    assert t.pool == 9 and [s.cuda_stream for s in t.told] == [7]
    t = nv._made(0, _Stream(9), world, returned=False)
    assert t.pool == 9 and not t.told


def test_streams_of_other_devices_are_refused(world):
    with pytest.raises(ValueError, match="another device"):
        nv._made(0, _Stream(9, device=1), world)


def test_default_streams_of_other_devices_are_refused(world, monkeypatch):
    """Every device's default stream has the same handle."""
    called = []
    for use in (lambda s: nv._made(0, s, world), lambda s: nv._launch("call", lambda *a: called.append(a) or 0, 0, s)):
        with pytest.raises(ValueError, match="another device"):
            use(_Stream(7, device=1))
    monkeypatch.setattr(nv, "_current_device", lambda: 0)
    nv._launch("call", lambda *a: called.append(a) or 0, 0, _Stream(9), 1)
    nv._launch("call", lambda *a: called.append(a) or 0, 0, None, 2)
    assert called == [(1, 9), (2, 7)]
