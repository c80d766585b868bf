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


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _cache():
    return bf16(4, 16, 2, 64), bf16(4, 16, 2, 64)


def _cache8():
    pool = [torch.zeros(4, 16, 2, 64, dtype=torch.uint8) for _ in range(2)]
    return (*pool, torch.ones(4, 16, 2), torch.ones(4, 16, 2))


class _Plan:
    num_splits, max_part_rows = 1, 2
    part_q_start, part_q_len, part_o_start, part_kv_lens = i32(0), i32(2), i32(0), i32(16)
    part_kv_indptr, part_kv_indices = i32(0, 1), i32(0)
    suffix_kv_indptr, suffix_kv_indices, suffix_kv_lens = i32(0, 1, 2), i32(1, 2), i32(5, 6)


# name: (the call, allocations it makes, of which results)
CALLS = {
    "paged_gather": (lambda q, t, s: pkv.paged_gather(*_cache(), *t, 9, stream=s), 2, 2),
    "paged_decode": (lambda q, t, s: pkv.paged_decode(q, *_cache(), *t, 0.1, stream=s), 3, 2),
    "paged_decode_noalloc": (lambda q, t, s: pkv.paged_decode_noalloc(q, *_cache(), *t, 0.1, stream=s), 2, 2),
    "paged_extend": (lambda q, t, s: pkv.paged_extend(q, *_cache(), t[0], *t, 1, 0.1, stream=s), 3, 2),
    "merge_states": (lambda q, t, s: pkv.merge_states(q[None], torch.zeros(1, 2, 4), stream=s), 2, 2),
    "shared_prefix_attention": (lambda q, t, s: pkv.shared_prefix_attention(
        q, *_cache(), i32(0), i32(2), i32(0), i32(0, 1), i32(0), i32(16), 2, 0.1, q.clone(), stream=s), 1, 0),
    "cascade_decode": (lambda q, t, s: pkv.cascade_decode(q, *_cache(), _Plan, 0.1, stream=s), 6, 2),
    "rope_cos_sin_table": (lambda q, t, s: pkv.rope_cos_sin_table(8, 64, 1e4, device="cuda:0", stream=s), 1, 1),
    "rotary_cos_sin_table": (lambda q, t, s: pkv.rotary_cos_sin_table(8, 64, 1e4, device="cuda:0", stream=s), 1, 1),
    "paged_decode_fp8": (lambda q, t, s: pkv.paged_decode_fp8(q, *_cache8(), *t, 0.1, stream=s), 3, 2),
    "paged_tree_attention": (lambda q, t, s: pkv.paged_tree_attention(
        q, *_cache(), t[0], *t, torch.zeros(2, 1, dtype=torch.int32), 1, 0.1, stream=s), 3, 2),
    "tree_mask_from_parents": (lambda q, t, s: pkv.tree_mask_from_parents(i32(-1, -1), t[0], 1, stream=s), 1, 1),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_what_a_call_makes_belongs_to_its_stream(made, monkeypatch, name):
    """Workspaces, which are dropped when the call returns, and results, which the caller's stream reads."""
    log, calls = made
    read_by = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "the caller's")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: read_by.append(stream))
    call, allocations, results = CALLS[name]
    q, table = bf16(2, 4, 64), (i32(0, 1, 2), i32(0, 1), i32(5, 6))
    log.clear()
    call(q, table, Side())
    mine = [at for fn, at in log if at is not None]
    assert mine == [SIDE] * allocations, log
    assert calls and all(stream == SIDE for _, stream in calls)
    assert read_by == ["the caller's"] * results
