"""Python binding of libpagedkv (attention over a paged KV pool on GB300).

Argument marshalling only: every function here checks that the tensors it is given have the
dtype, device and contiguity the C ABI expects, passes their device pointers and the current
CUDA stream to the matching ``pkv_*`` entry point, and turns a non-OK status into an exception.
All computation happens in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
a missing library is an error.

Names follow the C ABI in ``include/pagedkv.h`` (``pkv_kv_append`` -> ``kv_append`` ...).

A call with ``stream=s`` is the call under ``torch.cuda.stream(s)``: the results and workspaces that
it makes itself are allocated there, since the caching allocator orders the uses of a block by the
stream that it came from.  Inputs, and what the caller passes in, the caller orders against ``s``.
"""

from __future__ import annotations

import contextlib
import ctypes
import importlib
import math
import os
from typing import Optional, Tuple

import torch

__all__ = [
    "load", "library_path", "PagedKVError", "kv_append", "paged_gather", "decode_workspace_size",
    "paged_decode", "paged_decode_noalloc", "extend_workspace_size", "paged_extend",
    "merge_states", "shared_prefix_workspace_size", "shared_prefix_attention", "cascade_decode",
    "status_string", "version", "selftest_bounded_wait", "validate_page_table", "validate_slots",
    "rope_cos_sin_table", "rope_kv_append", "rotary_kv_append", "rotary_cos_sin_table",
    "kv_append_fp8", "rotary_kv_append_fp8", "paged_gather_fp8",
    "decode_fp8_workspace_size", "paged_decode_fp8",
    "kv_append_fp4", "rotary_kv_append_fp4", "paged_gather_fp4", "decode_fp4_workspace_size", "paged_decode_fp4",
    "copy_pages", "validate_page_copies", "compact_accepted",
    "tree_workspace_size", "paged_tree_attention", "tree_mask_from_parents", "DEVERR_PAGE_OOB", "DEVERR_SLOT_OOB", "DEVERR_LENGTH",
    "DEVERR_TIMEOUT", "DEVERR_INTERNAL", "DEVERR_ROW_OOB",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpagedkv.so")
_lib = None

DEVERR_PAGE_OOB = 0x1
DEVERR_SLOT_OOB = 0x2
DEVERR_LENGTH = 0x4
DEVERR_TIMEOUT = 0x8
DEVERR_INTERNAL = 0x10
DEVERR_ROW_OOB = 0x20

_c_i32, _c_i64, _c_f32, _c_sz, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p


class Pool(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("num_pages", _c_i64), ("page_size", _c_i32),
                ("num_kv_heads", _c_i32), ("head_dim", _c_i32)]


class CascadeSizes(ctypes.Structure):
    _fields_ = [("num_splits", _c_i32), ("num_parts", _c_i32), ("max_part_rows", _c_i32),
                ("num_part_indices", _c_i32), ("num_suffix_indices", _c_i32)]


class PoolFP8(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("num_pages", _c_i64),
                ("page_size", _c_i32), ("num_kv_heads", _c_i32), ("head_dim", _c_i32)]


class PoolFP4(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("num_pages", _c_i64),
                ("page_size", _c_i32), ("num_kv_heads", _c_i32), ("head_dim", _c_i32), ("k_global", _c_f32),
                ("v_global", _c_f32)]


class Plane(ctypes.Structure):
    _fields_ = [("base", _vp), ("slot_bytes", _c_i64)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", _c_i32), ("factor", ctypes.c_double), ("original_max_position", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("attention_factor", ctypes.c_double)]


class PagedKVError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libpagedkv.so (built by ``paged_kv_attention_10_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run paged_kv_attention_10_gb300.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER(Pool)
    P8 = ctypes.POINTER(PoolFP8)
    P4 = ctypes.POINTER(PoolFP4)
    PL = ctypes.POINTER(Plane)
    sig = {
        "pkv_status_string": (ctypes.c_char_p, [_c_i32]),
        "pkv_version": (_c_i32, []),
        "pkv_kv_append": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "pkv_paged_gather": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _vp, _vp, _vp, _vp]),
        "pkv_decode_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_paged_decode": (_c_i32, [P, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp, _vp,
                                      _c_sz, _vp, _vp]),
        "pkv_paged_decode_ctas": (_c_i32, [P, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp,
                                           _vp, _c_sz, _vp, _c_i32, _vp]),
        "pkv_paged_decode_l2keep": (_c_i32, [P, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp,
                                             _vp, _c_sz, _vp, _c_i32, _vp, _vp]),
        "pkv_extend_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_paged_extend": (_c_i32, [P, _vp, _c_i32, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_i32,
                                      _c_f32, _vp, _vp, _vp, _c_sz, _vp, _vp]),
        "pkv_merge_states": (_c_i32, [_vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32, _vp, _vp, _vp]),
        "pkv_merge_states_bf16": (_c_i32, [_vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32, _vp, _vp, _vp]),
        "pkv_shared_prefix_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_shared_prefix_attention": (_c_i32, [P, _vp, _c_i32, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _vp,
                                                 _vp, _c_i32, _c_f32, _vp, _vp, _c_i32, _vp, _c_sz, _vp,
                                                 _vp]),
        "pkv_rope_kv_append": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _c_i32, _vp, _c_i32, _c_i32, _vp, _vp]),
        "pkv_paged_decode_noalloc": (_c_i32, [P, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp,
                                              _vp, _vp]),
        "pkv_selftest_bounded_wait": (_c_i32, [_vp, _vp]),
        "pkv_validate_page_table": (_c_i32, [_vp, _vp, _vp, _c_i32, _c_i64, _c_i32, _c_i32, _vp]),
        "pkv_validate_slots": (_c_i32, [_vp, _c_i32, _c_i64, _vp]),
        "pkv_rope_cos_sin_table": (_c_i32, [_vp, _c_i32, _c_i32, ctypes.c_double, _vp]),
        "pkv_plan_shared_prefix": (_c_i32, [_vp, _vp, _vp, _c_i32, _vp, _vp, _c_i32, _c_i32, _c_i32,
                                            _c_i32, _c_i32, _c_i32, _c_i32, ctypes.POINTER(CascadeSizes),
                                            _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32,
                                            _c_i32]),
        "pkv_rotary_kv_append": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp, _vp,
                                          _c_i32, _c_i32, _vp, _vp]),
        "pkv_rotary_cos_sin_table": (_c_i32, [_vp, _c_i32, _c_i32, ctypes.c_double,
                                              ctypes.POINTER(RopeScaling), _vp]),
        "pkv_kv_append_fp8": (_c_i32, [P8, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "pkv_rotary_kv_append_fp8": (_c_i32, [P8, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp,
                                              _vp, _c_i32, _c_i32, _vp, _vp]),
        "pkv_decode_fp8_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_paged_decode_fp8": (_c_i32, [P8, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp, _vp,
                                          _c_sz, _vp, _c_i32, _vp]),
        "pkv_tree_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_paged_tree_attention": (_c_i32, [P, _vp, _c_i32, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _vp,
                                              _c_i32, _c_i32, _c_f32, _vp, _vp, _vp, _c_sz, _vp, _vp]),
        "pkv_tree_mask_from_parents": (_c_i32, [_vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32, _vp, _vp, _vp]),
        "pkv_paged_gather_fp8": (_c_i32, [P8, _vp, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp, _vp, _vp]),
        "pkv_kv_append_fp4": (_c_i32, [P4, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "pkv_rotary_kv_append_fp4": (_c_i32, [P4, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp,
                                              _vp, _c_i32, _c_i32, _vp, _vp]),
        "pkv_paged_gather_fp4": (_c_i32, [P4, _vp, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp, _vp, _vp]),
        "pkv_decode_fp4_workspace_size": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
        "pkv_paged_decode_fp4": (_c_i32, [P4, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _c_f32, _vp, _vp, _vp,
                                          _c_sz, _vp, _c_i32, _vp]),
        "pkv_copy_pages": (_c_i32, [PL, _c_i32, _c_i64, _c_i32, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "pkv_validate_page_copies": (_c_i32, [_vp, _vp, _c_i32, _c_i64, _vp]),
        "pkv_compact_accepted": (_c_i32, [PL, _c_i32, _c_i64, _c_i32, _vp, _vp, _vp, _c_i32, _vp, _vp,
                                          _c_i32, _vp, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


class _CheckedInPython:
    """Stands for the _checked module where it is not built: no call is taken."""

    def __getattr__(self, name):
        return lambda *args: None


_checked = None


def _load_checked():
    """The _checked module (csrc/binding.cpp): the once-a-layer calls, checked and made without Python."""
    global _checked
    load()
    try:
        _checked = importlib.import_module("._checked", __package__)
        if _checked.torch_version != str(torch.__version__):  # it reads the tensors of the torch it was built with
            _checked = _CheckedInPython()
    except ImportError:
        _checked = _CheckedInPython()
    return _checked


def _host_i(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous host {dtype} tensor")
    return t


def validate_page_table(kv_indptr, kv_indices, kv_lens, num_pages: int, page_size: int,
                        min_len: int = 1) -> None:
    """Check host page-table metadata before it goes to the device; raises PagedKVError naming
    the first bad request (``.bad``)."""
    _host_i(kv_indptr, "kv_indptr", torch.int32)
    _host_i(kv_indices, "kv_indices", torch.int32)
    _host_i(kv_lens, "kv_lens", torch.int32)
    B = kv_lens.numel()
    if kv_indptr.numel() != B + 1:
        raise ValueError("kv_indptr must have batch_size + 1 entries")
    bad = ctypes.c_int32(-1)
    st = load().pkv_validate_page_table(_ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_lens), B,
                                        int(num_pages), int(page_size), int(min_len), ctypes.byref(bad))
    if st != 0:
        e = PagedKVError(f"pkv_validate_page_table (request {bad.value})", st)
        e.bad = bad.value
        raise e


def validate_slots(slot_mapping, num_slots: int) -> None:
    """Check a host slot mapping (in range, no slot twice); raises PagedKVError naming the first
    bad token (``.bad``)."""
    _host_i(slot_mapping, "slot_mapping", torch.int64)
    bad = ctypes.c_int32(-1)
    st = load().pkv_validate_slots(_ptr(slot_mapping), slot_mapping.numel(), int(num_slots),
                                   ctypes.byref(bad))
    if st != 0:
        e = PagedKVError(f"pkv_validate_slots (token {bad.value})", st)
        e.bad = bad.value
        raise e


def validate_page_copies(src_pages, dst_pages, num_pages: int) -> None:
    """Check host lists of page copies (in range, no page a target twice or a target and another copy's source);
    raises PagedKVError naming the first bad copy (``.bad``)."""
    _host_i(src_pages, "src_pages", torch.int32)
    _host_i(dst_pages, "dst_pages", torch.int32)
    if src_pages.numel() != dst_pages.numel():
        raise ValueError("src_pages and dst_pages must have as many entries")
    bad = ctypes.c_int32(-1)
    st = load().pkv_validate_page_copies(_ptr(src_pages), _ptr(dst_pages), dst_pages.numel(), int(num_pages),
                                         ctypes.byref(bad))
    if st != 0:
        e = PagedKVError(f"pkv_validate_page_copies (copy {bad.value})", st)
        e.bad = bad.value
        raise e


def selftest_bounded_wait(err_word, stream=None) -> None:
    """Run the bounded-wait check: a GPU wait that nothing completes gives up after its limit and
    ORs DEVERR_TIMEOUT into err_word (int32 [1] on the device)."""
    _need(err_word, "err_word", torch.int32)
    dev = err_word.device
    with torch.cuda.device(dev):
        _call("pkv_selftest_bounded_wait", _ptr(err_word), _stream_ptr(stream, dev))


def status_string(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


def version() -> int:
    return int(load().pkv_version())


# ---------------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------------
def _need(t: torch.Tensor, name: str, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(stream, device):
    """Makes a call's own stream current, for what the call allocates or fills itself."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    return torch.cuda.stream(stream)


def _scratch(nbytes, device, stream):
    """A workspace that the caller did not bring.  It goes back to the allocator when the call returns, which
    may hand it on only behind the call: a block of the call's own stream."""
    with _on_stream(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _result(shape, dtype, device, stream, make=None):
    """A result that the caller did not bring (its values from `make`, torch.empty by default): of the call's
    stream, and read on the caller's current one."""
    make = make or torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with _on_stream(stream, device):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _pool(k_pool: torch.Tensor, v_pool: torch.Tensor) -> Pool:
    _need(k_pool, "k_pool", torch.bfloat16)
    _need(v_pool, "v_pool", torch.bfloat16, k_pool.device)
    if k_pool.dim() != 4 or k_pool.shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must both be [num_pages, page_size, num_kv_heads, head_dim]")
    n, ps, hkv, d = k_pool.shape
    return Pool(k_pool.data_ptr(), v_pool.data_ptr(), n, ps, hkv, d)


def _call(fn: str, *args):
    st = getattr(load(), fn)(*args)
    if st != 0:
        raise PagedKVError(fn, st)


# ---------------------------------------------------------------------------------------------
# operations
# ---------------------------------------------------------------------------------------------
def kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, err_word=None, stream=None) -> None:
    """Write k_new[t], v_new[t] into pool slot slot_mapping[t] (negative = skip). In place."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(k_new, "k_new", torch.bfloat16, dev)
    _need(v_new, "v_new", torch.bfloat16, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    T = slot_mapping.numel()
    if k_new.shape != (T, pool.num_kv_heads, pool.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [num_tokens, num_kv_heads, head_dim]")
    with torch.cuda.device(dev):
        _call("pkv_kv_append", ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T,
              _ptr(err_word), _stream_ptr(stream, dev))


def rope_cos_sin_table(max_position: int, head_dim: int, theta: float, device=None, out=None,
                       stream=None) -> torch.Tensor:
    """The fp32 [max_position, head_dim] cos/sin table rope_kv_append reads (row p: cos of the
    angles p * theta^(-2i/D), then their sines), computed by the library on ``device`` (default:
    the current CUDA device).  Built once, like a model's rotary buffer."""
    dev = torch.device(device) if device is not None else torch.device("cuda")
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if out is None:
        out = _result((max_position, head_dim), torch.float32, dev, stream)
    _need(out, "out", torch.float32, dev)
    if out.shape != (max_position, head_dim):
        raise ValueError("out must be [max_position, head_dim]")
    with torch.cuda.device(dev):
        _call("pkv_rope_cos_sin_table", _ptr(out), int(max_position), int(head_dim), float(theta),
              _stream_ptr(stream, dev))
    return out


def rope_kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, positions, cos_sin, q=None,
                   err_word=None, stream=None) -> None:
    """Rotate k_new (and q in place) by their positions and write K/V into the pool slots."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(k_new, "k_new", torch.bfloat16, dev)
    _need(v_new, "v_new", torch.bfloat16, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    _need(positions, "positions", torch.int32, dev)
    _need(cos_sin, "cos_sin", torch.float32, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    T = slot_mapping.numel()
    if k_new.shape != (T, pool.num_kv_heads, pool.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [num_tokens, num_kv_heads, head_dim]")
    if positions.numel() != T or cos_sin.dim() != 2 or cos_sin.shape[1] != pool.head_dim:
        raise ValueError("positions must be [num_tokens] and cos_sin [max_position, head_dim]")
    Hq = 0
    if q is not None:
        _need(q, "q", torch.bfloat16, dev)
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != pool.head_dim:
            raise ValueError("q must be [num_tokens, num_q_heads, head_dim]")
        Hq = q.shape[1]
    with torch.cuda.device(dev):
        _call("pkv_rope_kv_append", ctypes.byref(pool), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
              _ptr(positions), _ptr(cos_sin), cos_sin.shape[0], _ptr(q), Hq, T, _ptr(err_word),
              _stream_ptr(stream, dev))


def paged_gather(k_pool, v_pool, kv_indptr, kv_indices, kv_lens, total_len: int, err_word=None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Every request's K/V rows in position order, concatenated: [total_len, Hkv, D] each."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    for t, n in ((kv_indptr, "kv_indptr"), (kv_indices, "kv_indices"), (kv_lens, "kv_lens")):
        _need(t, n, torch.int32, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    B = kv_lens.numel()
    k_out, v_out = (_result((total_len, pool.num_kv_heads, pool.head_dim), torch.bfloat16, dev, stream)
                    for _ in range(2))
    with torch.cuda.device(dev):
        _call("pkv_paged_gather", ctypes.byref(pool), _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_lens),
              B, _ptr(k_out), _ptr(v_out), _ptr(err_word), _stream_ptr(stream, dev))
    return k_out, v_out


def decode_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_decode_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim))


def paged_decode(q, k_pool, v_pool, kv_indptr, kv_indices, kv_lens, sm_scale: float, out=None,
                 lse=None, workspace=None, err_word=None, stream=None, return_lse=True, max_ctas=0,
                 l2_keep_tokens=None):
    """Decode attention of q [B, Hq, D] over each request's paged KV. Returns (out, lse).
    ``max_ctas`` > 0 runs it on at most that many SMs (the rest stay free for other streams).
    ``l2_keep_tokens`` (int32 [B] on the device): request b's first l2_keep_tokens[b] positions
    are kept in L2 ahead of the rest (a prefix other requests of the batch share); the results
    do not change."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(q, "q", torch.bfloat16, dev)
    for t, n in ((kv_indptr, "kv_indptr"), (kv_indices, "kv_indices"), (kv_lens, "kv_lens")):
        _need(t, n, torch.int32, dev)
    B, Hq, D = q.shape
    if out is None:
        out = _result(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", torch.bfloat16, dev)
    if lse is None and return_lse:
        lse = _result((B, Hq), torch.float32, dev, stream)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    with torch.cuda.device(dev):
        need = int(load().pkv_decode_workspace_size(B, Hq, pool.num_kv_heads, D))
        if workspace is None:
            workspace = _scratch(max(need, 256), dev, stream)
        _need(workspace, "workspace", torch.uint8, dev)
        if l2_keep_tokens is not None:
            _need(l2_keep_tokens, "l2_keep_tokens", torch.int32, dev)
            if l2_keep_tokens.shape != (B,):
                raise ValueError("l2_keep_tokens must be [batch_size]")
            _call("pkv_paged_decode_l2keep", ctypes.byref(pool), _ptr(q), B, Hq, _ptr(kv_indptr),
                  _ptr(kv_indices), _ptr(kv_lens), float(sm_scale), _ptr(out), _ptr(lse),
                  _ptr(workspace), workspace.numel(), _ptr(err_word), int(max_ctas),
                  _ptr(l2_keep_tokens), _stream_ptr(stream, dev))
        elif max_ctas:
            _call("pkv_paged_decode_ctas", ctypes.byref(pool), _ptr(q), B, Hq, _ptr(kv_indptr),
                  _ptr(kv_indices), _ptr(kv_lens), float(sm_scale), _ptr(out), _ptr(lse),
                  _ptr(workspace), workspace.numel(), _ptr(err_word), int(max_ctas),
                  _stream_ptr(stream, dev))
        else:
            _call("pkv_paged_decode", ctypes.byref(pool), _ptr(q), B, Hq, _ptr(kv_indptr),
                  _ptr(kv_indices), _ptr(kv_lens), float(sm_scale), _ptr(out), _ptr(lse),
                  _ptr(workspace), workspace.numel(), _ptr(err_word), _stream_ptr(stream, dev))
    return out, lse


def paged_decode_noalloc(q, k_pool, v_pool, kv_indptr, kv_indices, kv_lens, sm_scale: float,
                         out=None, lse=None, err_word=None, stream=None, return_lse=True):
    """paged_decode with the split partials in the library's own device scratch (no workspace
    argument, nothing allocated per call). Returns (out, lse)."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(q, "q", torch.bfloat16, dev)
    for t, n in ((kv_indptr, "kv_indptr"), (kv_indices, "kv_indices"), (kv_lens, "kv_lens")):
        _need(t, n, torch.int32, dev)
    B, Hq, D = q.shape
    if out is None:
        out = _result(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", torch.bfloat16, dev)
    if lse is None and return_lse:
        lse = _result((B, Hq), torch.float32, dev, stream)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    with torch.cuda.device(dev):
        _call("pkv_paged_decode_noalloc", ctypes.byref(pool), _ptr(q), B, Hq, _ptr(kv_indptr),
              _ptr(kv_indices), _ptr(kv_lens), float(sm_scale), _ptr(out), _ptr(lse), _ptr(err_word),
              _stream_ptr(stream, dev))
    return out, lse


def extend_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim, max_extend_len,
                          device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_extend_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim,
                                                    max_extend_len))


def paged_extend(q, k_pool, v_pool, qo_indptr, kv_indptr, kv_indices, prefix_lens,
                 max_extend_len: int, sm_scale: float, out=None, lse=None, workspace=None,
                 err_word=None, stream=None, return_lse=True):
    """Ragged extend attention with a cached-prefix causal offset. Returns (out, lse)."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(q, "q", torch.bfloat16, dev)
    for t, n in ((qo_indptr, "qo_indptr"), (kv_indptr, "kv_indptr"), (kv_indices, "kv_indices"),
                 (prefix_lens, "prefix_lens")):
        _need(t, n, torch.int32, dev)
    N, Hq, D = q.shape
    B = prefix_lens.numel()
    if out is None:
        out = _result(q.shape, torch.bfloat16, dev, stream)
    _need(out, "out", torch.bfloat16, dev)
    if lse is None and return_lse:
        lse = _result((N, Hq), torch.float32, dev, stream)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    with torch.cuda.device(dev):
        need = int(load().pkv_extend_workspace_size(B, Hq, pool.num_kv_heads, D, max_extend_len))
        if workspace is None and need > 0:
            workspace = _scratch(need, dev, stream)
        if workspace is not None:
            _need(workspace, "workspace", torch.uint8, dev)
        _call("pkv_paged_extend", ctypes.byref(pool), _ptr(q), N, _ptr(qo_indptr), B, Hq, _ptr(kv_indptr),
              _ptr(kv_indices), _ptr(prefix_lens), int(max_extend_len), float(sm_scale), _ptr(out),
              _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel(),
              _ptr(err_word), _stream_ptr(stream, dev))
    return out, lse


def merge_states(o_parts, lse_parts, out=None, lse=None, stream=None):
    """LSE merge of split partials o_parts [S, N, H, D] (fp32 or bf16), lse_parts [S, N, H] fp32."""
    dev = o_parts.device
    bf16 = o_parts.dtype == torch.bfloat16
    fn = "pkv_merge_states_bf16" if bf16 else "pkv_merge_states"
    _need(o_parts, "o_parts", torch.bfloat16 if bf16 else torch.float32)
    _need(lse_parts, "lse_parts", torch.float32, dev)
    S, N, H, D = o_parts.shape
    if lse_parts.shape != (S, N, H):
        raise ValueError("lse_parts must be [S, N, H]")
    if out is None:
        out = _result((N, H, D), torch.bfloat16, dev, stream)
    if lse is None:
        lse = _result((N, H), torch.float32, dev, stream)
    _need(out, "out", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    with torch.cuda.device(dev):
        _call(fn, _ptr(o_parts), _ptr(lse_parts), S, N, H, D, _ptr(out), _ptr(lse),
              _stream_ptr(stream, dev))
    return out, lse


def shared_prefix_workspace_size(num_parts, num_q_heads, num_kv_heads, head_dim, max_part_rows,
                                 device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_shared_prefix_workspace_size(num_parts, num_q_heads, num_kv_heads,
                                                           head_dim, max_part_rows))


def shared_prefix_attention(q, k_pool, v_pool, q_start, q_len, o_start, kv_indptr, kv_indices,
                            kv_lens, max_part_rows: int, sm_scale: float, o_part, lse_part=None,
                            workspace=None, err_word=None, stream=None):
    """Unmasked attention of each part's query rows over the part's (shared) pages: the partial
    states of a cascade level, written at rows o_start[p].. of o_part (bf16) and lse_part."""
    pool = _pool(k_pool, v_pool)
    dev = k_pool.device
    _need(q, "q", torch.bfloat16, dev)
    for t, n in ((q_start, "q_start"), (q_len, "q_len"), (o_start, "o_start"), (kv_indptr, "kv_indptr"),
                 (kv_indices, "kv_indices"), (kv_lens, "kv_lens")):
        _need(t, n, torch.int32, dev)
    _need(o_part, "o_part", torch.bfloat16, dev)
    Nq, Hq, D = q.shape
    if o_part.dim() != 3 or o_part.shape[1:] != q.shape[1:]:
        raise ValueError("o_part must be [num_out_rows, num_q_heads, head_dim]")
    n_out = o_part.shape[0]
    if lse_part is not None:
        _need(lse_part, "lse_part", torch.float32, dev)
        if lse_part.shape != (n_out, Hq):
            raise ValueError("lse_part must be [num_out_rows, num_q_heads]")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32, dev)
    P = kv_lens.numel()
    with torch.cuda.device(dev):
        need = int(load().pkv_shared_prefix_workspace_size(P, Hq, pool.num_kv_heads, D, max_part_rows))
        if workspace is None and need > 0:
            workspace = _scratch(need, dev, stream)
        if workspace is not None:
            _need(workspace, "workspace", torch.uint8, dev)
        _call("pkv_shared_prefix_attention", ctypes.byref(pool), _ptr(q), Nq, _ptr(q_start), _ptr(q_len),
              _ptr(o_start), P, Hq, _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_lens), int(max_part_rows),
              float(sm_scale), _ptr(o_part), _ptr(lse_part), n_out, _ptr(workspace),
              0 if workspace is None else workspace.numel(), _ptr(err_word), _stream_ptr(stream, dev))
    return o_part, lse_part


def cascade_decode(q, k_pool, v_pool, plan, sm_scale: float, out=None, lse=None, o_parts=None,
                   lse_parts=None, prefix_workspace=None, decode_workspace=None, err_word=None,
                   stream=None):
    """Decode through a shared-prefix plan (``cascade.plan_shared_prefix``, its tensors on the
    device): the shared-prefix states, the decode over each request's own pages into the last
    split, and their log-sum-exp merge.  Three library calls on one stream; returns (out, lse)."""
    dev = q.device
    B, Hq, D = q.shape
    S = plan.num_splits
    with _on_stream(stream, dev):
        if o_parts is None:
            o_parts = torch.empty((S + 1, B, Hq, D), dtype=torch.bfloat16, device=dev)
        if lse_parts is None:
            lse_parts = torch.empty((S + 1, B, Hq), dtype=torch.float32, device=dev)
    if o_parts.shape != (S + 1, B, Hq, D) or lse_parts.shape != (S + 1, B, Hq):
        raise ValueError("o_parts / lse_parts must be [num_splits + 1, B, Hq, (D)]")
    shared_prefix_attention(q, k_pool, v_pool, plan.part_q_start, plan.part_q_len, plan.part_o_start,
                            plan.part_kv_indptr, plan.part_kv_indices, plan.part_kv_lens,
                            plan.max_part_rows, sm_scale, o_parts.view(-1, Hq, D),
                            lse_parts.view(-1, Hq), workspace=prefix_workspace, err_word=err_word,
                            stream=stream)
    paged_decode(q, k_pool, v_pool, plan.suffix_kv_indptr, plan.suffix_kv_indices, plan.suffix_kv_lens,
                 sm_scale, out=o_parts[S], lse=lse_parts[S], workspace=decode_workspace,
                 err_word=err_word, stream=stream)
    return merge_states(o_parts, lse_parts, out=out, lse=lse, stream=stream)


# ---------------------------------------------------------------------------------------------
# rotary append, 8-bit cache
# ---------------------------------------------------------------------------------------------
# Small steps are bound by the host, so each of these calls first goes to the _checked module, which checks the
# plain case and makes the call (None: it did neither).  What it does not take is checked here, with a few
# attribute reads a tensor; one that fails goes through _need, which says why.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_E4M3 = torch.float8_e4m3fn
_CODES = tuple(t for t in (_U8, getattr(torch, "float4_e2m1fn_x2", None)) if t is not None)


def _addr(t, name, dtype, index):
    """The address of a contiguous tensor of the given type on CUDA device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype, torch.device("cuda", index))
    return t.data_ptr()


def _addr_or_none(t, name, dtype, index):
    return None if t is None else _addr(t, name, dtype, index)


def _device_index(t, name):
    """The CUDA device index of the tensor that the others have to be beside."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


def _run(index, stream, fn: str, *args):
    """Call the library on device `index`'s current stream (or the given one); the device is made
    current only when it is not."""
    f = getattr(_lib if _lib is not None else load(), fn)
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current() == index:
        st = f(*args, raw)
    else:
        with torch.cuda.device(index):
            st = f(*args, raw)
    if st != 0:
        raise PagedKVError(fn, st)


def _done(status, fn) -> bool:
    """Whether the _checked module has made the call."""
    if status:
        raise PagedKVError(fn, status)
    return status is not None


def _pool_bf16(k_pool, v_pool):
    """(pool, its device index, its shape) of a bf16 cache."""
    index = _device_index(k_pool, "k_pool")
    k, v = _addr(k_pool, "k_pool", _BF16, index), _addr(v_pool, "v_pool", _BF16, index)
    shape = k_pool.shape
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must both be [num_pages, page_size, num_kv_heads, head_dim]")
    return Pool(k, v, *shape), index, shape


def _pool_fp8(k_pool, v_pool, k_scale, v_scale):
    """(pool, its device index, its shape) of an 8-bit cache."""
    if isinstance(k_pool, torch.Tensor) and k_pool.dtype not in (_E4M3, _U8):
        raise TypeError(f"k_pool must be torch.float8_e4m3fn (or its bytes as torch.uint8), got {k_pool.dtype}")
    index = _device_index(k_pool, "k_pool")
    k, v = _addr(k_pool, "k_pool", k_pool.dtype, index), _addr(v_pool, "v_pool", k_pool.dtype, index)
    ks, vs = _addr(k_scale, "k_scale", _F32, index), _addr(v_scale, "v_scale", _F32, index)
    shape = k_pool.shape
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must both be [num_pages, page_size, num_kv_heads, head_dim]")
    if k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
        raise ValueError("k_scale and v_scale must both be [num_pages, page_size, num_kv_heads]")
    return PoolFP8(k, v, ks, vs, *shape), index, shape


def _pool_fp4(k_pool, v_pool, k_scale, v_scale, k_global, v_global):
    """(pool, its device index, its shape in values) of a 4-bit cache."""
    for t, name, types, what in ((k_pool, "k_pool", _CODES, "torch.uint8 (two codes a byte)"),
                                 (k_scale, "k_scale", (_E4M3, _U8), "torch.float8_e4m3fn (or its bytes as torch.uint8)")):
        if isinstance(t, torch.Tensor) and t.dtype not in types:
            raise TypeError(f"{name} must be {what}, got {t.dtype}")
    index = _device_index(k_pool, "k_pool")
    k, v = _addr(k_pool, "k_pool", k_pool.dtype, index), _addr(v_pool, "v_pool", k_pool.dtype, index)
    _device_index(k_scale, "k_scale")
    ks, vs = _addr(k_scale, "k_scale", k_scale.dtype, index), _addr(v_scale, "v_scale", k_scale.dtype, index)
    shape = k_pool.shape
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must both be [num_pages, page_size, num_kv_heads, head_dim / 2]")
    if k_scale.shape != (*shape[:3], shape[3] // 8) or v_scale.shape != k_scale.shape or shape[3] % 8:
        raise ValueError("k_scale and v_scale must both be [num_pages, page_size, num_kv_heads, head_dim / 16]")
    shape = (*shape[:3], 2 * shape[3])
    return PoolFP4(k, v, ks, vs, *shape, k_global, v_global), index, shape


def _new_rows(index, shape, k_new, v_new, slot_mapping):
    """Check the new rows of an append: their addresses, the slots' and the number of tokens."""
    at = (_addr(k_new, "k_new", _BF16, index), _addr(v_new, "v_new", _BF16, index),
          _addr(slot_mapping, "slot_mapping", _I64, index))
    T = slot_mapping.numel()
    if k_new.shape != (T, shape[2], shape[3]) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [num_tokens, num_kv_heads, head_dim]")
    return at, T


def _rotary(fn, pool, index, shape, k_new, v_new, slot_mapping, positions, cos_sin, q, q_out, interleaved,
            err_word, stream):
    rows, T = _new_rows(index, shape, k_new, v_new, slot_mapping)
    pos, table = _addr(positions, "positions", _I32, index), _addr(cos_sin, "cos_sin", _F32, index)
    if positions.numel() != T or cos_sin.dim() != 2:
        raise ValueError("positions must be [num_tokens] and cos_sin [max_position, rotary_dim]")
    max_position, rotary_dim = cos_sin.shape
    if rotary_dim % 2 or not 2 <= rotary_dim <= shape[3]:
        raise ValueError("cos_sin's rotary_dim must be even and at most head_dim")
    q_at = out_at = None
    Hq = 0
    if q is not None:
        q_at = _addr(q, "q", _BF16, index)
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != shape[3]:
            raise ValueError("q must be [num_tokens, num_q_heads, head_dim]")
        out_at = q_at if q_out is None else _addr(q_out, "q_out", _BF16, index)
        if q_out is not None and q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        Hq = q.shape[1]
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _run(index, stream, fn, pool, *rows, pos, table, max_position, rotary_dim, 1 if interleaved else 0, q_at, out_at,
         Hq, T, _addr_or_none(err_word, "err_word", _I32, index))


def rotary_kv_append(k_pool, v_pool, k_new, v_new, slot_mapping, positions, cos_sin, q=None, q_out=None,
                     interleaved: bool = False, err_word=None, stream=None) -> None:
    """Rotate k_new (and q into q_out, in place when q_out is None) by their positions and write K/V
    into the pool slots.  The first cos_sin.shape[1] values of each head are rotated, in half-split
    or (``interleaved``) neighbouring pairs; negative slots are padding."""
    if _done((_checked or _load_checked()).rotary_kv_append(
            k_pool, v_pool, k_new, v_new, slot_mapping, positions, cos_sin, q, q_out, bool(interleaved), err_word,
            None if stream is None else stream.cuda_stream), "pkv_rotary_kv_append"):
        return
    pool, index, shape = _pool_bf16(k_pool, v_pool)
    _rotary("pkv_rotary_kv_append", pool, index, shape, k_new, v_new, slot_mapping, positions, cos_sin, q, q_out,
            interleaved, err_word, stream)


def rotary_kv_append_fp8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, positions, cos_sin,
                         q=None, q_out=None, interleaved: bool = False, err_word=None, stream=None) -> None:
    """rotary_kv_append into an 8-bit cache: K (rotated) and V quantised to e4m3 as they are written,
    with a power-of-two scale per row and head."""
    if _done((_checked or _load_checked()).rotary_kv_append_fp8(
            k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, positions, cos_sin, q, q_out,
            bool(interleaved), err_word, None if stream is None else stream.cuda_stream), "pkv_rotary_kv_append_fp8"):
        return
    pool, index, shape = _pool_fp8(k_pool, v_pool, k_scale, v_scale)
    _rotary("pkv_rotary_kv_append_fp8", pool, index, shape, k_new, v_new, slot_mapping, positions, cos_sin, q,
            q_out, interleaved, err_word, stream)


_ROPE_SCALING = {"none": 0, "linear": 1, "banded": 2, "yarn": 3}


def rotary_cos_sin_table(max_position: int, rotary_dim: int, theta: float, scaling: str = "none",
                         factor: float = 1.0, original_max_position: float = 0.0,
                         low: Optional[float] = None, high: Optional[float] = None,
                         attention_factor: Optional[float] = None, device=None, out=None,
                         stream=None) -> torch.Tensor:
    """The fp32 [max_position, rotary_dim] cos/sin table rotary_kv_append reads, with the frequencies
    scaled for long contexts: "none", "linear" (divided by factor), "banded" (low/high turns over the
    original context, 1 and 4 by default) or "yarn" (beta_slow/beta_fast, 1 and 32 by default;
    attention_factor 0.1 ln(factor) + 1 by default).  Built once, like a model's rotary buffer."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}")
    if low is None:
        low = 1.0
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if attention_factor is None:
        attention_factor = 0.1 * math.log(factor) + 1.0 if factor > 0 else 1.0
    spec = RopeScaling(_ROPE_SCALING[scaling], float(factor), float(original_max_position), float(low),
                       float(high), float(attention_factor))
    dev = torch.device(device) if device is not None else torch.device("cuda")
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if out is None:
        out = _result((max_position, rotary_dim), torch.float32, dev, stream)
    _need(out, "out", torch.float32, dev)
    if out.shape != (max_position, rotary_dim):
        raise ValueError("out must be [max_position, rotary_dim]")
    _run(dev.index, stream, "pkv_rotary_cos_sin_table", out.data_ptr(), int(max_position), int(rotary_dim),
         float(theta), spec)
    return out


def kv_append_fp8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word=None,
                  stream=None) -> None:
    """Quantise k_new[t], v_new[t] to e4m3 with a power-of-two scale per row and head and write them
    into pool slot slot_mapping[t] (negative = skip)."""
    if _done((_checked or _load_checked()).kv_append_fp8(
            k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, err_word,
            None if stream is None else stream.cuda_stream), "pkv_kv_append_fp8"):
        return
    pool, index, shape = _pool_fp8(k_pool, v_pool, k_scale, v_scale)
    rows, T = _new_rows(index, shape, k_new, v_new, slot_mapping)
    _run(index, stream, "pkv_kv_append_fp8", pool, *rows, T, _addr_or_none(err_word, "err_word", _I32, index))


def paged_gather_fp8(k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, out_indptr, k_out,
                     v_out, err_word=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read an 8-bit cache back as bf16: position j of request b goes to row out_indptr[b] + j of
    k_out/v_out [num_out_rows, num_kv_heads, head_dim]; other rows are left as they were."""
    if _done((_checked or _load_checked()).paged_gather_fp8(
            k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, out_indptr, k_out, v_out, err_word,
            None if stream is None else stream.cuda_stream), "pkv_paged_gather_fp8"):
        return k_out, v_out
    pool, index, shape = _pool_fp8(k_pool, v_pool, k_scale, v_scale)
    _gather("pkv_paged_gather_fp8", pool, index, shape, kv_indptr, kv_indices, kv_lens, out_indptr, k_out, v_out,
            err_word, stream)
    return k_out, v_out


def decode_fp8_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_decode_fp8_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim))


def _attention_io(q, index, head_dim, out, lse, return_lse, stream):
    """Check (or make) the outputs of an attention call over q [N, Hq, D]: (out, lse, the addresses of
    q, out and lse)."""
    at = _addr(q, "q", _BF16, index)
    if q.dim() != 3 or q.shape[2] != head_dim:
        raise ValueError("q must be [num_rows, num_q_heads, head_dim], with the pool's head_dim")
    if out is None:
        out = _result(q.shape, _BF16, q.device, stream)
    o_at = _addr(out, "out", _BF16, index)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if lse is None and return_lse:
        lse = _result(q.shape[:2], _F32, q.device, stream)
    l_at = _addr_or_none(lse, "lse", _F32, index)
    if lse is not None and lse.shape != q.shape[:2]:
        raise ValueError("lse must be [num_rows, num_q_heads]")
    return out, lse, at, o_at, l_at


def _page_table(index, kv_indptr, kv_indices, B):
    if kv_indptr.numel() != B + 1:
        raise ValueError("kv_indptr must have batch_size + 1 entries")
    return _addr(kv_indptr, "kv_indptr", _I32, index), _addr(kv_indices, "kv_indices", _I32, index)


def _decode_quant(fn, workspace_size, pool, index, shape, q, kv_indptr, kv_indices, kv_lens, sm_scale, out, lse, workspace,
                  err_word, stream, return_lse, max_ctas):
    lens = _addr(kv_lens, "kv_lens", _I32, index)
    B = kv_lens.numel()
    indptr, indices = _page_table(index, kv_indptr, kv_indices, B)
    out, lse, q_at, o_at, l_at = _attention_io(q, index, shape[3], out, lse, return_lse, stream)
    if q.shape[0] != B:
        raise ValueError("q must have one row per request")
    Hq = q.shape[1]
    if workspace is None:
        need = workspace_size(B, Hq, shape[2], shape[3], index)
        workspace = _scratch(max(need, 256), q.device, stream)
    _run(index, stream, fn, pool, q_at, B, Hq, indptr, indices, lens, sm_scale, o_at, l_at,
         _addr(workspace, "workspace", _U8, index), workspace.numel(), _addr_or_none(err_word, "err_word", _I32, index),
         max_ctas)
    return out, lse


def paged_decode_fp8(q, k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, sm_scale: float,
                     out=None, lse=None, workspace=None, err_word=None, stream=None, return_lse=True,
                     max_ctas=0):
    """Decode attention of q [B, Hq, D] over each request's pages of an 8-bit cache.  Returns
    (out, lse); arguments as for paged_decode."""
    if out is not None and workspace is not None and (lse is not None or not return_lse) and _done(
            (_checked or _load_checked()).paged_decode_fp8(
                k_pool, v_pool, k_scale, v_scale, q, out, lse, kv_indptr, kv_indices, kv_lens, sm_scale, workspace,
                err_word, max_ctas, None if stream is None else stream.cuda_stream), "pkv_paged_decode_fp8"):
        return out, lse
    pool, index, shape = _pool_fp8(k_pool, v_pool, k_scale, v_scale)
    return _decode_quant("pkv_paged_decode_fp8", decode_fp8_workspace_size, pool, index, shape, q, kv_indptr,
                         kv_indices, kv_lens, sm_scale, out, lse, workspace, err_word, stream, return_lse, max_ctas)


def kv_append_fp4(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, k_global: float = 1.0,
                  v_global: float = 1.0, err_word=None, stream=None) -> None:
    """Quantise k_new[t], v_new[t] to e2m1 with an e4m3 scale for every 16 values (and the cache's own scales k_global,
    v_global) and write them into pool slot slot_mapping[t] (negative = skip).  k_pool and v_pool are
    uint8 [num_pages, page_size, num_kv_heads, head_dim / 2], k_scale and v_scale float8_e4m3fn [..., head_dim / 16].
    k_global and v_global belong to the cache: every call on it, of any kind, has to be given the same two (nothing in the
    cache tells a call that left one out); 1.0 is for a cache whose calls all leave them out."""
    if _done((_checked or _load_checked()).kv_append_fp4(
            k_pool, v_pool, k_scale, v_scale, k_global, v_global, k_new, v_new, slot_mapping, err_word,
            None if stream is None else stream.cuda_stream), "pkv_kv_append_fp4"):
        return
    pool, index, shape = _pool_fp4(k_pool, v_pool, k_scale, v_scale, k_global, v_global)
    rows, T = _new_rows(index, shape, k_new, v_new, slot_mapping)
    _run(index, stream, "pkv_kv_append_fp4", pool, *rows, T, _addr_or_none(err_word, "err_word", _I32, index))


def rotary_kv_append_fp4(k_pool, v_pool, k_scale, v_scale, k_new, v_new, slot_mapping, positions, cos_sin,
                         q=None, q_out=None, interleaved: bool = False, k_global: float = 1.0, v_global: float = 1.0,
                         err_word=None, stream=None) -> None:
    """rotary_kv_append into a 4-bit cache: K (rotated) and V quantised as by kv_append_fp4, with the cache's own k_global and
    v_global as there."""
    if _done((_checked or _load_checked()).rotary_kv_append_fp4(
            k_pool, v_pool, k_scale, v_scale, k_global, v_global, k_new, v_new, slot_mapping, positions, cos_sin, q,
            q_out, bool(interleaved), err_word, None if stream is None else stream.cuda_stream),
            "pkv_rotary_kv_append_fp4"):
        return
    pool, index, shape = _pool_fp4(k_pool, v_pool, k_scale, v_scale, k_global, v_global)
    _rotary("pkv_rotary_kv_append_fp4", pool, index, shape, k_new, v_new, slot_mapping, positions, cos_sin, q,
            q_out, interleaved, err_word, stream)


def _gather(fn, pool, index, shape, kv_indptr, kv_indices, kv_lens, out_indptr, k_out, v_out, err_word, stream):
    at = [_addr(t, n, _I32, index) for t, n in ((kv_indptr, "kv_indptr"), (kv_indices, "kv_indices"),
                                                (kv_lens, "kv_lens"), (out_indptr, "out_indptr"))]
    ko, vo = _addr(k_out, "k_out", _BF16, index), _addr(v_out, "v_out", _BF16, index)
    B = kv_lens.numel()
    if kv_indptr.numel() != B + 1 or out_indptr.numel() != B + 1:
        raise ValueError("kv_indptr and out_indptr must have batch_size + 1 entries")
    if k_out.dim() != 3 or k_out.shape[1:] != shape[2:] or v_out.shape != k_out.shape:
        raise ValueError("k_out/v_out must be [num_out_rows, num_kv_heads, head_dim]")
    _run(index, stream, fn, pool, *at[:3], B, at[3], k_out.shape[0], ko, vo,
         _addr_or_none(err_word, "err_word", _I32, index))


def paged_gather_fp4(k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, out_indptr, k_out,
                     v_out, k_global: float = 1.0, v_global: float = 1.0, err_word=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read a 4-bit cache back as bf16: position j of request b goes to row out_indptr[b] + j of
    k_out/v_out [num_out_rows, num_kv_heads, head_dim]; other rows are left as they were.  k_global and v_global are those that
    the cache was written with."""
    if _done((_checked or _load_checked()).paged_gather_fp4(
            k_pool, v_pool, k_scale, v_scale, k_global, v_global, kv_indptr, kv_indices, kv_lens, out_indptr, k_out,
            v_out, err_word, None if stream is None else stream.cuda_stream), "pkv_paged_gather_fp4"):
        return k_out, v_out
    pool, index, shape = _pool_fp4(k_pool, v_pool, k_scale, v_scale, k_global, v_global)
    _gather("pkv_paged_gather_fp4", pool, index, shape, kv_indptr, kv_indices, kv_lens, out_indptr, k_out, v_out,
            err_word, stream)
    return k_out, v_out


def decode_fp4_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_decode_fp4_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim))


def paged_decode_fp4(q, k_pool, v_pool, k_scale, v_scale, kv_indptr, kv_indices, kv_lens, sm_scale: float,
                     out=None, lse=None, workspace=None, k_global: float = 1.0, v_global: float = 1.0, err_word=None,
                     stream=None, return_lse=True, max_ctas=0):
    """Decode attention of q [B, Hq, D] over each request's pages of a 4-bit cache.  Returns
    (out, lse); arguments as for paged_decode, and the k_global and v_global that the cache was written with."""
    if out is not None and workspace is not None and (lse is not None or not return_lse) and _done(
            (_checked or _load_checked()).paged_decode_fp4(
                k_pool, v_pool, k_scale, v_scale, k_global, v_global, q, out, lse, kv_indptr, kv_indices, kv_lens,
                sm_scale, workspace, err_word, max_ctas, None if stream is None else stream.cuda_stream),
            "pkv_paged_decode_fp4"):
        return out, lse
    pool, index, shape = _pool_fp4(k_pool, v_pool, k_scale, v_scale, k_global, v_global)
    return _decode_quant("pkv_paged_decode_fp4", decode_fp4_workspace_size, pool, index, shape, q, kv_indptr,
                         kv_indices, kv_lens, sm_scale, out, lse, workspace, err_word, stream, return_lse, max_ctas)


# ---------------------------------------------------------------------------------------------
# movements of rows within a cache
# ---------------------------------------------------------------------------------------------
def _planes(tensors):
    """(planes, how many, the device index, num_pages, page_size) of a cache's tensors [num_pages, page_size, ...]."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("tensors must name at least one tensor of the cache")
    index = _device_index(tensors[0], "tensors[0]")
    planes = (Plane * len(tensors))()
    for i, t in enumerate(tensors):
        at = _addr(t, f"tensors[{i}]", t.dtype if isinstance(t, torch.Tensor) else None, index)
        if t.dim() < 2 or t.shape[:2] != tensors[0].shape[:2] or not t.numel():
            raise ValueError("tensors must all be [num_pages, page_size, ...], with the same num_pages and page_size")
        planes[i] = Plane(at, t.numel() * t.element_size() // (t.shape[0] * t.shape[1]))
    return planes, len(tensors), index, tensors[0].shape[0], tensors[0].shape[1]


def copy_pages(tensors, src_pages, dst_pages, rows=None, err_word=None, stream=None) -> None:
    """Copy page src_pages[i] (its first rows[i] rows where rows is given) to page dst_pages[i] (negative = skip) in
    every one of the cache's tensors [num_pages, page_size, ...]: K, V and scales of a layer or of all layers, of any type, at
    most 256, no two over the same memory.  No page may be a target twice, or a target and another copy's source
    (validate_page_copies)."""
    if _done((_checked or _load_checked()).copy_pages(
            tensors, src_pages, dst_pages, rows, err_word, None if stream is None else stream.cuda_stream),
            "pkv_copy_pages"):
        return
    planes, count, index, num_pages, page_size = _planes(tensors)
    src, dst = _addr(src_pages, "src_pages", _I32, index), _addr(dst_pages, "dst_pages", _I32, index)
    n = dst_pages.numel()
    if src_pages.numel() != n or (rows is not None and rows.numel() != n):
        raise ValueError("src_pages, dst_pages and rows must have as many entries")
    _run(index, stream, "pkv_copy_pages", planes, count, num_pages, page_size, src, dst,
         _addr_or_none(rows, "rows", _I32, index), n, _addr_or_none(err_word, "err_word", _I32, index))


def compact_accepted(tensors, kv_indptr, kv_indices, prefix_lens, accepted_indptr, accepted, err_word=None,
                     stream=None) -> None:
    """Move the accepted tokens of drafted trees behind their prefix in every one of the cache's tensors (as for
    copy_pages): the row at position prefix_lens[b] + accepted[accepted_indptr[b] + k] of request b goes to position
    prefix_lens[b] + k.  A request's accepted indices ascend."""
    if _done((_checked or _load_checked()).compact_accepted(
            tensors, kv_indptr, kv_indices, prefix_lens, accepted_indptr, accepted, err_word,
            None if stream is None else stream.cuda_stream), "pkv_compact_accepted"):
        return
    planes, count, index, num_pages, page_size = _planes(tensors)
    prefix = _addr(prefix_lens, "prefix_lens", _I32, index)
    B = prefix_lens.numel()
    indptr, indices = _page_table(index, kv_indptr, kv_indices, B)
    starts, taken = _addr(accepted_indptr, "accepted_indptr", _I32, index), _addr(accepted, "accepted", _I32, index)
    if accepted_indptr.numel() != B + 1:
        raise ValueError("accepted_indptr must have batch_size + 1 entries")
    _run(index, stream, "pkv_compact_accepted", planes, count, num_pages, page_size, indptr, indices, prefix, B, starts,
         taken, accepted.numel(), _addr_or_none(err_word, "err_word", _I32, index))


# ---------------------------------------------------------------------------------------------
# trees of drafted tokens
# ---------------------------------------------------------------------------------------------
def tree_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim, max_tree_len, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(load().pkv_tree_workspace_size(batch_size, num_q_heads, num_kv_heads, head_dim,
                                                  max_tree_len))


def _mask_words(tree_mask, index, rows, max_tree_len):
    at = _addr(tree_mask, "tree_mask", _I32, index)
    if tree_mask.dim() != 2 or tree_mask.shape[0] != rows or 32 * tree_mask.shape[1] < max_tree_len:
        raise ValueError("tree_mask must be [num_q_tokens, words] with 32 * words >= max_tree_len")
    return at, tree_mask.shape[1]


def paged_tree_attention(q, k_pool, v_pool, qo_indptr, kv_indptr, kv_indices, prefix_lens, tree_mask,
                         max_tree_len: int, sm_scale: float, out=None, lse=None, workspace=None,
                         err_word=None, stream=None, return_lse=True):
    """Attention of each request's drafted tokens (rows qo_indptr[b].. of q) over its cached prefix
    and the drafted tokens whose bits its tree_mask row (int32 [num_q_tokens, words]) sets.  Returns
    (out, lse)."""
    if out is not None and workspace is not None and (lse is not None or not return_lse) and _done(
            (_checked or _load_checked()).paged_tree_attention(
                k_pool, v_pool, q, out, lse, qo_indptr, kv_indptr, kv_indices, prefix_lens, tree_mask, max_tree_len,
                sm_scale, workspace, err_word, None if stream is None else stream.cuda_stream),
            "pkv_paged_tree_attention"):
        return out, lse
    pool, index, shape = _pool_bf16(k_pool, v_pool)
    qo, prefix = _addr(qo_indptr, "qo_indptr", _I32, index), _addr(prefix_lens, "prefix_lens", _I32, index)
    B = prefix_lens.numel()
    indptr, indices = _page_table(index, kv_indptr, kv_indices, B)
    if qo_indptr.numel() != B + 1:
        raise ValueError("qo_indptr must have batch_size + 1 entries")
    out, lse, q_at, o_at, l_at = _attention_io(q, index, shape[3], out, lse, return_lse, stream)
    N, Hq, D = q.shape
    mask, words = _mask_words(tree_mask, index, N, max_tree_len)
    if workspace is None:
        need = tree_workspace_size(B, Hq, shape[2], D, max_tree_len, index)
        workspace = _scratch(max(need, 256), q.device, stream)
    _run(index, stream, "pkv_paged_tree_attention", pool, q_at, N, qo, B, Hq, indptr, indices, prefix, mask, words,
         max_tree_len, sm_scale, o_at, l_at, _addr(workspace, "workspace", _U8, index), workspace.numel(),
         _addr_or_none(err_word, "err_word", _I32, index))
    return out, lse


def tree_mask_from_parents(parents, qo_indptr, max_tree_len: int, out=None, err_word=None,
                           stream=None) -> torch.Tensor:
    """The tree_mask of trees given by parents (int32 [num_tokens], each the parent's index within its
    request's tree, negative for a root; parents come before their children)."""
    index = _device_index(parents, "parents")
    at, qo = _addr(parents, "parents", _I32, index), _addr(qo_indptr, "qo_indptr", _I32, index)
    if parents.dim() != 1 or qo_indptr.numel() < 1:
        raise ValueError("parents must be [num_tokens] and qo_indptr [batch_size + 1]")
    N = parents.numel()
    if out is None:
        # zeroed on the call's stream, before the kernel
        out = _result((N, -(-int(max_tree_len) // 32)), _I32, parents.device, stream, torch.zeros)
    mask, words = _mask_words(out, index, N, max_tree_len)
    _run(index, stream, "pkv_tree_mask_from_parents", at, qo, qo_indptr.numel() - 1, N, max_tree_len, words, mask,
         _addr_or_none(err_word, "err_word", _I32, index))
    return out
