"""Refusals of the rotary append, the 8-bit cache and the tree attention that need no GPU: the C ABI
on arguments it checks before it touches CUDA, and the binding on tensors it does not take."""

import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
SOME = ctypes.c_void_p(0x10000)  # an aligned address that is never read
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_attention_10_gb300 import build

    build.build()
    import paged_kv_attention_10_gb300 as p

    return p


@pytest.fixture(scope="module")
def lib(pkv):
    return pkv.load()


def _pool(pkv, D=64, Hkv=2, pages=4, ps=16, k=SOME):
    return ctypes.byref(pkv.Pool(k, SOME, pages, ps, Hkv, D))


def _pool8(pkv, D=64, Hkv=2, pages=4, ps=16, k=SOME, scale=SOME):
    return ctypes.byref(pkv.PoolFP8(k, SOME, scale, SOME, pages, ps, Hkv, D))


def _rotary(pool, fn, k=SOME, v=SOME, slots=SOME, pos=SOME, table=SOME, most=16, R=64, q=SOME, q_out=SOME, Hq=4,
            T=3):
    return fn(pool, k, v, slots, pos, table, most, R, 0, q, q_out, Hq, T, None, None)


@pytest.mark.parametrize("name,pool", [("pkv_rotary_kv_append", _pool), ("pkv_rotary_kv_append_fp8", _pool8)])
def test_rotary_append_refusals(pkv, lib, name, pool):
    fn = getattr(lib, name)
    good = pool(pkv)
    assert _rotary(good, fn, T=0) == OK  # nothing to write: nothing is launched
    assert _rotary(None, fn) == INVALID
    assert _rotary(pool(pkv, k=ODD), fn) == INVALID
    assert _rotary(pool(pkv, D=60), fn) == INVALID
    assert _rotary(good, fn, T=-1) == INVALID
    for R in (0, -2, 63, 66):
        assert _rotary(good, fn, R=R) == INVALID
    assert _rotary(good, fn, most=0) == INVALID
    for missing in ("k", "v", "slots", "pos", "table"):
        assert _rotary(good, fn, **{missing: None}) == INVALID
    for odd in ("k", "v", "table", "q", "q_out"):
        assert _rotary(good, fn, **{odd: ODD}) == INVALID
    assert _rotary(good, fn, q=None) == INVALID            # heads without Q
    assert _rotary(good, fn, q_out=None) == INVALID
    assert _rotary(good, fn, Hq=0) == INVALID              # Q without heads
    # Q and its rotated copy overlap: 3 tokens * 4 heads * 64 values * 2 bytes = 1536 bytes
    assert _rotary(good, fn, q_out=ctypes.c_void_p(0x10000 + 1520)) == INVALID
    assert _rotary(good, fn, q=ctypes.c_void_p(0x10010)) == INVALID
    assert _rotary(pool(pkv, D=264), fn, R=64) == UNSUPPORTED
    assert _rotary(good, fn, T=1 << 30) == UNSUPPORTED


def test_8_bit_pool_refusals(pkv, lib):
    f = lib.pkv_kv_append_fp8
    good = _pool8(pkv)
    assert f(good, SOME, SOME, SOME, 0, None, None) == OK
    assert f(None, SOME, SOME, SOME, 1, None, None) == INVALID
    assert f(_pool8(pkv, scale=None), SOME, SOME, SOME, 1, None, None) == INVALID
    assert f(_pool8(pkv, scale=ODD), SOME, SOME, SOME, 1, None, None) == INVALID
    assert f(_pool8(pkv, pages=0), SOME, SOME, SOME, 1, None, None) == INVALID
    assert f(good, ODD, SOME, SOME, 1, None, None) == INVALID
    assert f(good, SOME, SOME, None, 1, None, None) == INVALID
    assert f(_pool8(pkv, D=512), SOME, SOME, SOME, 1, None, None) == UNSUPPORTED
    g = lib.pkv_paged_gather_fp8
    a = [SOME] * 3
    assert g(good, *a, 0, SOME, 4, SOME, SOME, None, None) == OK
    assert g(good, *a, 2, SOME, 0, SOME, SOME, None, None) == OK
    assert g(None, *a, 2, SOME, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, -1, SOME, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, SOME, -4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, None, 4, SOME, SOME, None, None) == INVALID
    assert g(good, *a, 2, SOME, 4, ODD, SOME, None, None) == INVALID
    assert g(good, None, SOME, SOME, 2, SOME, 4, SOME, SOME, None, None) == INVALID


def test_table_refusals(pkv, lib):
    f = lib.pkv_rotary_cos_sin_table

    def call(most=16, R=64, theta=1e4, table=None, **s):
        spec = pkv.RopeScaling(s.get("kind", 0), s.get("factor", 2.0), s.get("orig", 4096.0), s.get("low", 1.0),
                               s.get("high", 4.0), s.get("att", 1.0))
        return f(table, most, R, theta, ctypes.byref(spec) if s else None, None)

    inf, nan = float("inf"), float("nan")
    assert call(most=0) == OK
    for kind in (1, 2, 3):
        assert call(most=0, kind=kind) == OK
    assert call() == INVALID  # no table
    assert call(most=-1) == INVALID
    for R in (0, 63, -2):
        assert call(most=0, R=R) == INVALID
    for theta in (0.0, -1.0, inf, nan):
        assert call(most=0, theta=theta) == INVALID
    for bad in (dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=nan),
                dict(kind=2, orig=0.0), dict(kind=2, low=0.0), dict(kind=2, low=4.0), dict(kind=3, high=inf),
                dict(kind=3, att=0.0), dict(kind=3, theta=1.0), dict(kind=3, orig=nan)):
        assert call(most=0, **bad) == INVALID, bad


def test_binding_refuses_host_tensors_and_wrong_types(pkv):
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    new = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.rotary_kv_append(k, k, new, new, slots, slots.int(), torch.zeros(8, 64))
    with pytest.raises(TypeError, match="e4m3"):
        pkv.kv_append_fp8(k, k, k, k, new, new, slots)
    k8 = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_fp8(k8, k8, k, k, new, new, slots)
    with pytest.raises(ValueError, match="scaling"):
        pkv.rotary_cos_sin_table(8, 64, 1e4, scaling="other")


def test_decode_fp8_refusals(pkv, lib):
    f = lib.pkv_paged_decode_fp8
    good = _pool8(pkv)

    def call(pool=good, q=SOME, B=2, Hq=4, indptr=SOME, out=SOME, ws=SOME, n=0, ctas=0):
        return f(pool, q, B, Hq, indptr, SOME, SOME, 1.0, out, None, ws, n, None, ctas, None)

    assert call(B=0) == OK
    assert call(pool=None) == INVALID
    assert call(B=-1) == INVALID
    assert call(Hq=0) == INVALID
    assert call(ctas=-1) == INVALID
    assert call(q=None) == INVALID and call(indptr=None) == INVALID and call(out=None) == INVALID
    assert call(q=ODD) == INVALID and call(out=ODD) == INVALID
    assert call(Hq=5) == INVALID                       # not a multiple of the KV heads
    assert call(Hq=34) == UNSUPPORTED                  # 17 query heads per KV head
    assert call(pool=_pool8(pkv, D=32)) == UNSUPPORTED
    assert call(B=1 << 30) == UNSUPPORTED


def test_tree_refusals(pkv, lib):
    f = lib.pkv_paged_tree_attention
    good = _pool(pkv)

    def call(pool=good, q=SOME, N=6, qo=SOME, B=2, Hq=4, mask=SOME, words=1, most=3, out=SOME, ws=SOME, n=0):
        return f(pool, q, N, qo, B, Hq, SOME, SOME, SOME, mask, words, most, 1.0, out, None, ws, n, None, None)

    assert call(B=0) == OK and call(N=0) == OK and call(most=0) == OK
    assert call(pool=None) == INVALID
    assert call(B=-1) == INVALID and call(N=-1) == INVALID and call(most=-1) == INVALID
    assert call(Hq=0) == INVALID and call(Hq=5) == INVALID
    assert call(words=-1) == INVALID
    assert call(most=33) == INVALID                    # one word holds 32 tokens
    for missing in ("q", "qo", "mask", "out"):
        assert call(**{missing: None}) == INVALID
    assert call(q=ODD) == INVALID and call(out=ODD) == INVALID
    assert call(pool=_pool(pkv, pages=1 << 28)) == UNSUPPORTED

    g = lib.pkv_tree_mask_from_parents
    assert g(SOME, SOME, 0, 4, 4, 1, SOME, None, None) == OK
    assert g(SOME, SOME, 1, 4, 33, 1, SOME, None, None) == INVALID
    assert g(None, SOME, 1, 4, 4, 1, SOME, None, None) == INVALID
    assert g(SOME, SOME, 1, -4, 4, 1, SOME, None, None) == INVALID
    assert g(SOME, SOME, 65536, 4, 4, 1, SOME, None, None) == UNSUPPORTED
    assert g(SOME, SOME, 1, 4, 1025, 33, SOME, None, None) == UNSUPPORTED
