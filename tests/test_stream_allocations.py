"""Where a call on a stream of its own allocates and fills what the caller left out: on that stream.
The caching allocator takes a block back, and hands it on, in the order of the stream that it was
allocated on, and a fill on another stream is ordered against nothing.  No GPU: the library, the streams
and the allocations are stand-ins that write down which stream was current."""

import contextlib

import pytest
import torch

import paged_kv_attention_10_gb300 as pkv

SIDE = 0x7700  # the side stream's handle


class Side:
    cuda_stream = SIDE


class Library:
    """Takes every call: sizes of 4096 bytes, status 0."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                return 4096
            stream = args[-1]
            self.calls.append((name, getattr(stream, "value", stream)))
            return 0

        return call


@pytest.fixture
def made(monkeypatch):
    """(allocations as (function, current stream's handle), library calls as (name, stream's handle))."""
    current, log, calls = [None], [], []

    @contextlib.contextmanager
    def on(stream):
        before = current[0]
        current[0] = stream.cuda_stream
        yield
        current[0] = before

    for name in ("empty", "zeros", "empty_like"):
        real = getattr(torch, name)

        def make(*args, _real=real, _name=name, **kw):
            log.append((_name, current[0]))
            kw.pop("device", None)
            return _real(*args, **kw)

        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Side() if handle == SIDE else None)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None)
    library = Library(calls)
    monkeypatch.setattr(pkv, "_lib", library)
    monkeypatch.setattr(pkv, "_checked", pkv._CheckedInPython())
    monkeypatch.setattr(pkv, "_current", lambda: 0)
    monkeypatch.setattr(pkv, "_need", lambda t, name, dtype, device=None: t)
    monkeypatch.setattr(pkv, "_device_index", lambda t, name: 0)
    monkeypatch.setattr(pkv, "_addr", lambda t, name, dtype, index: t.data_ptr())
    return log, calls


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_tree_mask_is_zeroed_on_the_calls_stream(made):
    log, calls = made
    parents, qo = i32(-1, 0, 0), i32(0, 3)
    log.clear()
    pkv.tree_mask_from_parents(parents, qo, 3, stream=Side())
    assert calls == [("pkv_tree_mask_from_parents", SIDE)]
    assert log == [("zeros", SIDE)]
