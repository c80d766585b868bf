"""Refusals of the 4-bit cache and of the movements of rows that need no GPU: the C ABI on arguments it
checks before it touches CUDA, and the binding on tensors it does not take."""

import ctypes
import math

import pytest
import torch

from test_stream_allocations import SIDE, Side, made  # noqa: F401
from test_operators_host import ODD, SOME, _rotary, INVALID, OK, UNSUPPORTED, pkv, lib  # noqa: F401


def _pool4(pkv, D=64, Hkv=2, pages=4, ps=16, k=SOME, scale=SOME, kg=1.0, vg=1.0):  # noqa: F811
    return ctypes.byref(pkv.PoolFP4(k, SOME, scale, SOME, pages, ps, Hkv, D, kg, vg))


def test_pool_refusals(pkv, lib):  # noqa: F811
    f = lib.pkv_kv_append_fp4
    good = _pool4(pkv)

    def call(pool=good, k=SOME, slots=SOME, T=1):
        return f(pool, k, SOME, slots, T, None, None)

    assert call(T=0) == OK
    assert call(pool=None) == INVALID
    for bad in (dict(scale=None), dict(k=None), dict(k=ODD), dict(pages=0), dict(ps=0), dict(Hkv=0),
                dict(D=0), dict(D=56), dict(D=-16)):
        assert call(_pool4(pkv, **bad)) == INVALID, bad
    for g in (0.0, -1.0, math.nan, math.inf, 2.0 ** -65, 2.0 ** 65):
        assert call(_pool4(pkv, kg=g)) == INVALID, g
        assert call(_pool4(pkv, vg=g), T=0) == INVALID, g
    assert call(_pool4(pkv, kg=2.0 ** -64, vg=2.0 ** 64), T=0) == OK
    assert call(k=ODD) == INVALID
    assert call(slots=None) == INVALID
    assert call(T=-1) == INVALID
    assert call(_pool4(pkv, D=512)) == UNSUPPORTED


def test_rotary_append_refusals(pkv, lib):  # noqa: F811
    fn = lib.pkv_rotary_kv_append_fp4
    good = _pool4(pkv)
    assert _rotary(good, fn, T=0) == OK
    assert _rotary(None, fn) == INVALID
    assert _rotary(_pool4(pkv, D=56), fn, R=56) == INVALID
    assert _rotary(good, fn, T=-1) == INVALID
    for R in (0, -2, 63, 66):
        assert _rotary(good, fn, R=R) == INVALID
    assert _rotary(good, fn, most=0) == INVALID
    for missing in ("k", "v", "slots", "pos", "table"):
        assert _rotary(good, fn, **{missing: None}) == INVALID
    for odd in ("k", "v", "table", "q", "q_out"):
        assert _rotary(good, fn, **{odd: ODD}) == INVALID
    assert _rotary(good, fn, q=None) == INVALID
    assert _rotary(good, fn, Hq=0) == INVALID
    assert _rotary(good, fn, q_out=ctypes.c_void_p(0x10000 + 1520)) == INVALID  # Q and its rotated copy overlap
    assert _rotary(_pool4(pkv, D=272), fn, R=64) == UNSUPPORTED
    assert _rotary(good, fn, T=1 << 30) == UNSUPPORTED


def test_gather_refusals(pkv, lib):  # noqa: F811
    g = lib.pkv_paged_gather_fp4
    good = _pool4(pkv)
    a = [SOME] * 3
    assert g(good, *a, 0, SOME, 4, SOME, SOME, None, None) == OK
    assert g(good, *a, 2, SOME, 0, SOME, SOME, None, None) == OK
    assert g(None, *a, 2, SOME, 4, SOME, SOME, None, None) == INVALID
    assert g(_pool4(pkv, vg=0.0), *a, 2, SOME, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, -1, SOME, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, SOME, -4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, None, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, SOME, 4, ODD, SOME, None, None) == INVALID
    assert g(good, None, SOME, SOME, 2, SOME, 4, SOME, SOME, None, None) == INVALID


def test_decode_refusals(pkv, lib):  # noqa: F811
    f = lib.pkv_paged_decode_fp4
    good = _pool4(pkv)

    def call(pool=good, q=SOME, B=2, Hq=4, indptr=SOME, out=SOME, ws=SOME, n=0, ctas=0):
        return f(pool, q, B, Hq, indptr, SOME, SOME, 1.0, out, None, ws, n, None, ctas, None)

    assert call(B=0) == OK
    assert call(pool=None) == INVALID
    assert call(pool=_pool4(pkv, kg=math.nan)) == INVALID
    assert call(B=-1) == INVALID
    assert call(Hq=0) == INVALID
    assert call(ctas=-1) == INVALID
    assert call(q=None) == INVALID and call(indptr=None) == INVALID and call(out=None) == INVALID
    assert call(q=ODD) == INVALID and call(out=ODD) == INVALID
    assert call(Hq=5) == INVALID                       # not a multiple of the KV heads
    assert call(Hq=34) == UNSUPPORTED                  # 17 query heads per KV head
    assert call(pool=_pool4(pkv, D=32)) == UNSUPPORTED
    assert call(B=1 << 30) == UNSUPPORTED


def _planes(pkv, *planes):  # noqa: F811
    return (pkv.Plane * len(planes))(*[pkv.Plane(b, n) for b, n in planes])


BASE = 0x10000


def test_copy_refusals(pkv, lib):  # noqa: F811
    f = lib.pkv_copy_pages
    good = _planes(pkv, (BASE, 64), (BASE, 8))

    def call(planes=good, count=2, pages=4, ps=16, src=SOME, dst=SOME, n=3):
        return f(planes, count, pages, ps, src, dst, None, n, None, None)

    assert call(n=0) == OK
    assert call(planes=None, count=0) == OK
    assert call(planes=None) == INVALID
    assert call(count=-1) == INVALID and call(pages=0) == INVALID and call(ps=0) == INVALID and call(n=-1) == INVALID
    assert call(src=None) == INVALID and call(dst=None) == INVALID
    for bad in ((None, 64), (BASE, 0), (BASE, -4)):
        assert call(planes=_planes(pkv, (BASE, 64), bad)) == INVALID, bad
    assert call(planes=_planes(pkv, (BASE, 64), (BASE, 1 << 27))) == UNSUPPORTED     # a page of 2^31 bytes
    assert call(planes=_planes(pkv, *[(BASE, 64)] * 257), count=257) == UNSUPPORTED
    assert call(planes=_planes(pkv, (BASE, 1 << 26)), count=1, n=1 << 30) == UNSUPPORTED


def test_compact_refusals(pkv, lib):  # noqa: F811
    f = lib.pkv_compact_accepted
    good = _planes(pkv, (BASE, 64), (BASE, 8))

    def call(planes=good, count=2, pages=4, ps=16, indptr=SOME, indices=SOME, prefix=SOME, B=2, starts=SOME,
             accepted=SOME, n=3):
        return f(planes, count, pages, ps, indptr, indices, prefix, B, starts, accepted, n, None, None)

    assert call(n=0) == OK and call(B=0) == OK and call(planes=None, count=0) == OK
    assert call(planes=None) == INVALID
    assert call(count=-1) == INVALID and call(pages=0) == INVALID and call(ps=0) == INVALID
    assert call(n=-1) == INVALID and call(B=-1) == INVALID
    for missing in ("indptr", "indices", "prefix", "starts", "accepted"):
        assert call(**{missing: None}) == INVALID
    assert call(planes=_planes(pkv, (None, 64)), count=1) == INVALID
    assert call(planes=_planes(pkv, *[(BASE, 64)] * 257), count=257) == UNSUPPORTED
    assert call(planes=_planes(pkv, (BASE, 1 << 26)), count=1, B=1 << 30) == UNSUPPORTED


@pytest.mark.parametrize("name", ["pkv_copy_pages", "pkv_compact_accepted"])
def test_tensors_that_share_memory_are_refused(pkv, lib, name):  # noqa: F811
    """The same tensor twice, one within another, one that begins on another's last byte, in any order; 4 pages of 16 slots."""
    pages = 4
    tail = [SOME, SOME, None, 1] if name == "pkv_copy_pages" else [SOME, SOME, SOME, 1, SOME, SOME, 1]
    for planes in ([(BASE, 64), (BASE, 64)], [(BASE, 64), (BASE + 1024, 1)], [(BASE + 4095, 8), (BASE, 64)],
                   [(BASE + 8192, 64), (BASE, 64), (BASE + 4096, 65)], [((1 << 64) - 4096, 65)]):
        assert getattr(lib, name)(_planes(pkv, *planes), len(planes), pages, 16, *tail, None, None) == INVALID, planes


def test_page_copies_are_validated(pkv):  # noqa: F811
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731

    def bad(src, dst, pages=8):
        try:
            pkv.validate_page_copies(i32(*src), i32(*dst), pages)
        except pkv.PagedKVError as e:
            return e.bad
        return None

    assert bad([], []) is None
    assert bad([0, 0, 1], [2, 3, 4]) is None        # one source, two targets
    assert bad([0, 9, 1], [2, -1, 4]) is None       # padding
    assert bad([0, 1], [2, 2]) == 1                 # a target twice
    assert bad([0, 2], [2, 3]) == 1                 # a target that is another copy's source
    assert bad([5, 1], [3, 5]) == 0
    assert bad([5], [5]) is None                    # onto itself
    assert bad([0, 8], [2, 3]) == 1 and bad([0, 1], [2, 8]) == 1 and bad([-1, 1], [2, 3]) == 0
    with pytest.raises(ValueError, match="entries"):
        pkv.validate_page_copies(i32(1), i32(2, 3), 8)
    with pytest.raises(TypeError, match="int32"):
        pkv.validate_page_copies(i32(1).long(), i32(2), 8)


def test_binding_refuses_host_tensors_and_wrong_types(pkv):  # noqa: F811
    codes = torch.zeros(2, 16, 2, 32, dtype=torch.uint8)
    scale = torch.zeros(2, 16, 2, 4, dtype=torch.float8_e4m3fn)
    new = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_fp4(codes, codes, scale, scale, new, new, slots)
    with pytest.raises(TypeError, match="uint8"):
        pkv.kv_append_fp4(new, new, scale, scale, new, new, slots)
    with pytest.raises(TypeError, match="e4m3"):
        pkv.kv_append_fp4(codes, codes, scale.float(), scale.float(), new, new, slots)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.rotary_kv_append_fp4(codes, codes, scale, scale, new, new, slots, slots.int(), torch.zeros(8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_gather_fp4(codes, codes, scale, scale, slots.int(), slots.int(), slots.int(), slots.int(), new, new)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_decode_fp4(new, codes, codes, scale, scale, slots.int(), slots.int(), slots.int(), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.copy_pages([codes], slots.int(), slots.int())
    with pytest.raises(TypeError, match="Tensor"):
        pkv.copy_pages([3], slots.int(), slots.int())
    with pytest.raises(ValueError, match="CUDA"):
        pkv.compact_accepted((codes,), slots.int(), slots.int(), slots.int(), slots.int(), slots.int())


def test_what_the_decode_makes_belongs_to_its_stream(pkv, made, monkeypatch):  # noqa: F811
    """Its workspace, which is dropped when the call returns, and its results, which the caller's stream reads."""
    log, calls = made
    read_by = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "the caller's")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: read_by.append(stream))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    pool = [torch.zeros(4, 16, 2, n, dtype=torch.uint8) for n in (32, 32, 4, 4)]
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    log.clear()
    pkv.paged_decode_fp4(q, *pool, i32(0, 1, 2), i32(0, 1), i32(5, 6), 0.1, stream=Side())
    assert [at for fn, at in log if at is not None] == [SIDE] * 3, log
    assert calls and all(stream == SIDE for _, stream in calls)
    assert read_by == ["the caller's"] * 2
