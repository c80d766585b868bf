"""Decode over the 8-bit cache against 64-bit attention over the values its bytes stand for.

Besides the bound of _attention64: a weight p_j vs_j is held in f16 relative to the largest of its row (up
to a factor of 2), so below 2^-14 of that it is off by up to 2^-25 of it instead of 2^-11 of itself.
That adds 2^-24 max_j(p_j vs_j) sum_j |v8_jd| to a result."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from _attention64 import attend, check

pytestmark = pytest.mark.gpu

F16 = 2.0 ** -11  # half a step: the weights of the second product are rounded to f16


def make(seed, lens, Hq, Hkv, D, page, scales="rows", spare=3):
    """A pool whose unowned slots, and every row behind a request's end, hold NaN bytes and huge scales."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + spare
    perm = rng.permutation(num_pages)[: sum(need)]
    indptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    codes = np.full((2, num_pages * page, Hkv, D), 0x7F, dtype=np.uint8)
    scale = np.full((2, num_pages * page, Hkv), 1e30, dtype=np.float32)
    rows = []
    for b, n in enumerate(lens):
        j = np.arange(n)
        slot = perm[indptr[b] + j // page].astype(np.int64) * page + j % page
        rows.append(slot)
        for at in range(2):
            x = rng.standard_normal((n, Hkv, D)) * np.exp(0.5 * rng.standard_normal((1, Hkv, D)))
            if scales == "wide" and at == 1:  # values of neighbouring rows differ by up to 2^40
                x *= 2.0 ** rng.integers(-20, 21, (n, Hkv, 1))
            c, s = cache8.quantise(x)
            if scales == "head":  # one scale per head, not a power of two
                s = np.broadcast_to(0.0123 * (1 + np.arange(Hkv)), (n, Hkv))
                c = cache8.e4m3_codes(np.clip(x / s[..., None], -448, 448))
            codes[at, slot], scale[at, slot] = c, s
    t = dict(indptr=indptr, pages=perm.astype(np.int32))
    dev = {k: torch.tensor(v).cuda() for k, v in t.items()}
    pool = [torch.tensor(codes[i].reshape(num_pages, page, Hkv, D)).cuda() for i in range(2)]
    pool += [torch.tensor(scale[i].reshape(num_pages, page, Hkv)).cuda() for i in range(2)]
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(len(lens), Hq, D, generator=gen).to(torch.bfloat16)
    return dict(pool=pool, q=q, codes=codes, scale=scale, rows=rows, sm=1 / math.sqrt(D), lens=lens, **dev)


def verify(s, out, lse, what=""):
    q = oracle.as_f64(s["q"])
    B, Hq, D = q.shape
    Hkv = s["codes"].shape[2]
    G = Hq // Hkv
    o = out.double().cpu().numpy()
    l = lse.double().cpu().numpy()
    for b, n in enumerate(s["lens"]):
        for h in range(Hkv):
            k, v = (cache8.e4m3_values(s["codes"][at, s["rows"][b], h])
                    * s["scale"][at, s["rows"][b], h].astype(np.float64)[:, None] for at in range(2))
            hs = slice(h * G, (h + 1) * G)
            ref = attend(q[b, hs], k, v, s["sm"])
            vs = s["scale"][1, s["rows"][b], h].astype(np.float64)
            v8 = np.abs(cache8.e4m3_values(s["codes"][1, s["rows"][b], h])).sum(0)
            extra = 2.0 ** -24 * (ref[4] * vs).max(-1)[:, None] * v8
            check(o[b, hs], l[b, hs], ref, n, F16, f"{what} request {b} head {h}", extra)


def decode(lib, s, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.paged_decode_fp8(s["q"].cuda(), *s["pool"], s["indptr"], s["pages"], s["lens_dev"] if "lens_dev" in s
                                    else torch.tensor(s["lens"], dtype=torch.int32).cuda(), s["sm"], err_word=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


SHAPES = [
    # lens, Hq, Hkv, D, page
    ((1,), 1, 1, 64, 16),
    ((1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65), 14, 2, 64, 16),
    ((37, 100, 256, 511), 14, 2, 64, 16),
    ((100, 640, 333), 16, 8, 128, 1),
    ((5, 700, 33, 1200), 32, 8, 128, 16),
    ((50, 4000), 32, 8, 128, 16),
    ((9, 129, 777), 28, 4, 128, 8),
    ((24, 25, 500), 6, 3, 64, 24),
    ((40, 1000), 40, 5, 128, 40),
    ((300, 2), 7, 7, 64, 32),
    ((5, 16, 1500), 16, 1, 128, 16),
    ((5, 1600), 8, 1, 64, 8),
    ((31, 32, 2, 1), 16, 16, 64, 64),
    ((257, 3), 48, 16, 128, 16),
    ((70, 600), 12, 6, 128, 3),
    ((100, 900), 32, 2, 128, 5),
    ((90, 250), 3, 1, 128, 1),
]


@pytest.mark.parametrize("scales", ["rows", "wide", "head"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1]}/{s[2]}-D{s[3]}-p{s[4]}")
def test_decode8(lib, shape, scales):
    lens, Hq, Hkv, D, page = shape
    s = make(sum(lens) + Hq, lens, Hq, Hkv, D, page, scales)
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("max_ctas", [1, 2, 7, 100])
def test_decode8_on_fewer_sms(lib, max_ctas):
    s = make(5, (1, 300, 47, 2000, 8), 32, 8, 128, 16)
    out, lse, err = decode(lib, s, max_ctas=max_ctas)
    assert err == 0
    verify(s, out, lse)


def test_many_short_requests(lib):
    rng = np.random.default_rng(3)
    s = make(6, tuple(rng.integers(1, 50, 300).tolist()), 8, 2, 64, 16)
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_queries_of_every_size(lib):
    """Rows of q near the ends of bf16's range, with a scale that makes their scores ordinary, rows with
    one value far above the rest, and rows of zeros."""
    s = make(7, (40, 100, 65, 33, 70), 8, 2, 128, 16)
    q = s["q"].float()
    q[0] *= 2.0 ** 90
    q[1] *= 2.0 ** -90
    q[2, :, 5] = 3.0e4
    q[3] = 0.0
    q[4, ::2] *= 2.0 ** -30
    s["q"] = q.to(torch.bfloat16)
    for b, sm in ((0, 2.0 ** -90), (1, 2.0 ** 90), (2, 1e-4), (3, 1.0), (4, 1.0)):
        one = dict(s, q=s["q"][b: b + 1], lens=s["lens"][b: b + 1], sm=sm, rows=s["rows"][b: b + 1],
                   indptr=s["indptr"][b: b + 2] - s["indptr"][b],
                   pages=s["pages"][int(s["indptr"][b]): int(s["indptr"][b + 1])])
        one["indptr"], one["pages"] = one["indptr"].contiguous(), one["pages"].contiguous()
        out, lse, err = decode(lib, one)
        assert err == 0
        verify(one, out, lse, f"q {b}")


def test_zero_rows_negative_scale_and_empty_requests(lib):
    s = make(8, (20, 64, 3), 4, 2, 64, 16)
    zero, tiny = cache8.quantise(np.zeros((64, 2, 64)))
    for at in range(2):  # the second request's K and V are rows of zeros
        s["codes"][at, s["rows"][1]], s["scale"][at, s["rows"][1]] = zero, tiny
        s["pool"][at].view(-1, 2, 64)[torch.tensor(s["rows"][1])] = torch.tensor(zero).cuda()
        s["pool"][2 + at].view(-1, 2)[torch.tensor(s["rows"][1])] = torch.tensor(tiny).float().cuda()
    s["sm"] = -0.3
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)
    assert torch.all(out[1] == 0)
    s["lens_dev"] = torch.tensor([20, 0, 3], dtype=torch.int32).cuda()
    out2, lse2, err = decode(lib, s)
    assert err == lib.DEVERR_LENGTH
    assert torch.all(out2[1] == 0) and torch.all(torch.isneginf(lse2[1]))
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[2], out[2])


def test_a_nan_in_one_request_stays_there(lib):
    s = make(9, (50, 60), 4, 2, 64, 16)
    s["pool"][1].view(-1, 2, 64)[int(s["rows"][0][7]), 1, 9] = 0x7F
    out, lse, err = decode(lib, s)
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    want[0, 2:, 9] = True
    assert torch.equal(nan, want) and not torch.isnan(lse).any()


def test_bad_pages_are_reported(lib):
    s = make(10, (40, 60), 4, 2, 64, 16)
    good = s["pages"].clone()
    for page, want in ((10 ** 6, lib.DEVERR_PAGE_OOB), (-1, lib.DEVERR_PAGE_OOB)):
        s["pages"] = good.clone()
        s["pages"][1] = page
        assert decode(lib, s)[2] == want
    s["pages"] = good
    ref = decode(lib, s)
    s["lens_dev"] = torch.tensor([49, 60], dtype=torch.int32).cuda()  # three pages hold 48 positions
    out, lse, err = decode(lib, s)
    assert err == lib.DEVERR_LENGTH and torch.equal(out[1], ref[0][1])


def test_deterministic_and_on_another_stream(lib):
    s = make(11, (900, 31, 4000, 77), 32, 8, 128, 16)
    out, lse, _ = decode(lib, s)
    st = torch.cuda.Stream()
    args = (s["q"].cuda(), *s["pool"], s["indptr"], s["pages"], torch.tensor(s["lens"], dtype=torch.int32).cuda(), s["sm"])
    torch.cuda.synchronize()
    for _ in range(3):
        o2, l2 = lib.paged_decode_fp8(*args, stream=st)
        st.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_shared_pages(lib):
    """Two requests that list the same pages."""
    s = make(12, (128, 100), 8, 2, 128, 16)
    s["pages"][8: 8 + 4] = s["pages"][:4]
    s["rows"][1][:64] = s["rows"][0][:64]
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_pool_past_32_bits(lib):
    """Slots whose byte offsets pass 4 GB, for the append, the decode (boxes and rows) and the read-back."""
    first = 280_000  # pages of 16 KB
    shape = (first + 20, 16, 8, 128)
    pool = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool += [torch.ones(shape[:3], device="cuda") for _ in range(2)]
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(300, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(1, 32, 128, generator=gen).to(torch.bfloat16).cuda()
    slots = first * 16 + torch.randperm(320, generator=gen)[:300].cuda()
    lib.kv_append_fp8(*pool, k, v, slots)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    flat = [pool[0].view(-1, 1, 8, 128), pool[1].view(-1, 1, 8, 128), pool[2].view(-1, 1, 8), pool[3].view(-1, 1, 8)]
    out, lse = lib.paged_decode_fp8(q, *flat, i32([0, 300]), slots.int(), i32([300]), 0.1)
    ref = {}
    for name, x in (("k", k), ("v", v)):
        codes, scale = cache8.quantise(oracle.as_f64(x))
        ref[name] = cache8.e4m3_values(codes) * scale[..., None]
    qd, o, l = oracle.as_f64(q)[0], oracle.as_f64(out)[0], oracle.as_f64(lse)[0]
    for h in range(8):
        a = attend(qd[4 * h: 4 * h + 4], ref["k"][:, h], ref["v"][:, h], 0.1)
        extra = 2.0 ** -24 * a[4].max(-1)[:, None] * 4 * np.abs(ref["v"][:, h]).sum(0)
        check(o[4 * h: 4 * h + 4], l[4 * h: 4 * h + 4], a, 300, F16, f"head {h}", extra)
    ko, vo = (torch.zeros(320, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = i32(list(range(first, first + 20)))
    lib.paged_gather_fp8(*pool, i32([0, 20]), pages, i32([320]), i32([0, 320]), ko, vo)
    assert np.array_equal(oracle.as_f64(ko[slots - first * 16]), ref["k"])
    assert np.array_equal(oracle.as_f64(vo[slots - first * 16]), ref["v"])
    # the same rows as pages of 16, in page order
    o16, l16 = lib.paged_decode_fp8(q, *pool, i32([0, 20]), pages, i32([320]), 0.1)
    small = [x[first:].contiguous() for x in pool]
    o2, l2 = lib.paged_decode_fp8(q, *small, i32([0, 20]), pages - first, i32([320]), 0.1)
    assert torch.equal(o16, o2) and torch.equal(l16, l2)
