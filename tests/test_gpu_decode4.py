"""Decode over the 4-bit cache against 64-bit attention over the values its codes stand for.

The bound is _attention64's with weights rounded to f16.  Besides, weights are held relative to one (2^8) that is at most
the row's largest, so one below 2^-22 of that is a subnormal f16 and off by up to 2^-33 of it: 2^-32 max_j(p_j) sum_j
|v_jd| is added to a result."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache4
from _attention64 import attend, check

pytestmark = pytest.mark.gpu

F16 = 2.0 ** -11  # half a step: the weights of the second product are rounded to f16
KG, VG = 0.0113, 0.00235


def make(seed, lens, Hq, Hkv, D, page, scales="rows", spare=3):
    """A pool whose unowned slots, and every row behind a request's end, have NaN scales."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + spare
    perm = rng.permutation(num_pages)[: sum(need)]
    indptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    codes = np.full((2, num_pages * page, Hkv, D // 2), 0x77, dtype=np.uint8)
    scale = np.full((2, num_pages * page, Hkv, D // 16), 0x7F, dtype=np.uint8)
    rows = []
    for b, n in enumerate(lens):
        j = np.arange(n)
        slot = perm[indptr[b] + j // page].astype(np.int64) * page + j % page
        rows.append(slot)
        for at, g in ((0, KG), (1, VG)):
            if scales == "any":  # every scale that is a number, V's over all 18 binades
                c = rng.integers(0, 256, (n, Hkv, D // 2)).astype(np.uint8)
                s = rng.integers(0, 0x50 if at == 0 else 0x7F, (n, Hkv, D // 16)).astype(np.uint8)
            else:
                x = rng.standard_normal((n, Hkv, D)) * np.exp(0.5 * rng.standard_normal((1, Hkv, D)))
                c, s = cache4.quantise(x, g)
            codes[at, slot], scale[at, slot] = c, s
    t = dict(indptr=indptr, pages=perm.astype(np.int32))
    dev = {k: torch.tensor(v).cuda() for k, v in t.items()}
    pool = [torch.tensor(x[i].reshape(num_pages, page, Hkv, -1)).cuda() for x in (codes, scale) for i in range(2)]
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
        k, v = (cache4.values(s["codes"][at, s["rows"][b]], s["scale"][at, s["rows"][b]], g)
                for at, g in ((0, KG), (1, VG)))
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            ref = attend(q[b, hs], k[:, h], v[:, h], s["sm"])
            extra = 2.0 ** -32 * ref[4].max(-1)[:, None] * np.abs(v[:, h]).sum(0)
            check(o[b, hs], l[b, hs], ref, n, F16, f"{what} request {b} head {h}", extra)


def decode(lib, s, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.paged_decode_fp4(s["q"].cuda(), *s["pool"], s["indptr"], s["pages"], s["lens_dev"] if "lens_dev" in s
                                    else torch.tensor(s["lens"], dtype=torch.int32).cuda(), s["sm"], err_word=err,
                                    k_global=KG, v_global=VG, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


SHAPES = [
    # lens, Hq, Hkv, D, page
    ((1,), 1, 1, 64, 16),
    ((1,), 1, 1, 128, 16),
    ((1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65), 14, 2, 64, 16),
    ((1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65), 14, 2, 128, 16),
    ((37, 100, 256, 511), 14, 2, 64, 16),
    ((100, 640, 333), 16, 8, 128, 1),
    ((5, 700, 33, 1200), 32, 8, 128, 16),
    ((50, 4000), 32, 8, 128, 16),
    ((9, 129, 777), 28, 4, 128, 8),
    ((24, 25, 500), 6, 3, 64, 24),
    ((40, 1000), 40, 5, 128, 40),
    ((40, 1000), 40, 5, 64, 7),
    ((300, 2), 7, 7, 64, 32),
    ((5, 16, 1500), 16, 1, 128, 16),
    ((5, 1600), 8, 1, 64, 8),
    ((5, 1600), 8, 1, 64, 3),
    ((31, 32, 2, 1), 16, 16, 64, 64),
    ((257, 3), 48, 16, 128, 16),
    ((70, 600), 12, 6, 128, 3),
    ((100, 900), 32, 2, 128, 5),
    ((90, 250), 3, 1, 128, 1),
    ((90, 250), 33, 11, 64, 16),
    ((90, 250), 33, 11, 128, 2),
    ((300, 250), 48, 3, 128, 16),
    ((300, 250), 9, 3, 64, 1),
]


@pytest.mark.parametrize("scales", ["rows", "any"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1]}/{s[2]}-D{s[3]}-p{s[4]}")
def test_decode4(lib, shape, scales):
    lens, Hq, Hkv, D, page = shape
    s = make(sum(lens) + Hq, lens, Hq, Hkv, D, page, scales)
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("max_ctas", [1, 2, 7, 100])
def test_decode4_on_fewer_sms(lib, max_ctas):
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


def test_scores_that_jump_within_a_request(lib):
    """The largest score comes first, last, or in the middle of a warp's positions, far above what was before."""
    for at in (0, 31, 32, 700, 1999):
        s = make(70 + at, (2000,), 8, 2, 128, 16)
        slot = s["rows"][0][at]
        s["scale"][0, slot] = 0x7E  # K of 448 times its codes
        s["pool"][2].view(-1, 2, 8)[int(slot)] = 0x7E
        out, lse, err = decode(lib, s)
        assert err == 0
        verify(s, out, lse, f"at {at}")


def test_zero_rows_negative_scale_and_empty_requests(lib):
    s = make(8, (20, 64, 3), 4, 2, 64, 16)
    for at in range(2):  # the second request's K and V are rows of zeros
        r = torch.tensor(s["rows"][1])
        s["scale"][at, s["rows"][1]] = 0
        s["pool"][2 + at].view(-1, 2, 4)[r] = 0
    s["sm"] = -0.3
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)
    assert torch.all(out[1] == 0)
    s["lens_dev"] = torch.tensor([20, 0, 3], dtype=torch.int32).cuda()
    out2, lse2, err = decode(lib, s)
    assert err == lib.DEVERR_LENGTH
    assert torch.all(out2[1] == 0) and torch.all(torch.isneginf(lse2[1]))
    assert torch.equal(out2[0], out[0]) and torch.equal(lse2[0], lse[0])
    assert torch.equal(out2[2], out[2]) and torch.equal(lse2[2], lse[2])


@pytest.mark.parametrize("lens", [(50, 60), (5000, 60)])  # the second: the request is split over CTAs
def test_nan_stays_in_its_request(lib, lens):
    s = make(9, lens, 4, 2, 64, 16)
    s["pool"][3].view(-1, 2, 4)[int(s["rows"][0][7]), 1, 2] = 0x7F  # V: one block of KV head 1
    out, lse, err = decode(lib, s)
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    want[0, 2:, 32:48] = True
    assert torch.equal(nan, want) and not torch.isnan(lse).any()
    s["pool"][3].view(-1, 2, 4)[int(s["rows"][0][7]), 1, 2] = 0x38
    s["pool"][2].view(-1, 2, 4)[int(s["rows"][0][40]), 0, 1] = 0x7F  # K: all of KV head 0's queries
    out, lse, err = decode(lib, s)
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    want[0, :2] = True
    assert torch.equal(nan, want)
    assert torch.equal(torch.isnan(lse).cpu(), want[:, :, 0])


def test_a_request_of_nothing_but_nan(lib):
    s = make(19, (33, 700), 4, 2, 128, 16)
    s["pool"][2].view(-1, 2, 8)[torch.tensor(s["rows"][0])] = 0x7F
    out, lse, err = decode(lib, s)
    assert err == 0
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert not torch.isnan(out[1]).any() and not torch.isnan(lse[1]).any()


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
        o2, l2 = lib.paged_decode_fp4(*args, k_global=KG, v_global=VG, stream=st)
        st.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("shape", [((100, 31), 8, 1, 64, 1), ((100, 700), 8, 2, 128, 16), ((100, 700), 32, 8, 128, 16),
                                   ((100, 700), 33, 11, 128, 16), ((90, 250), 9, 3, 64, 5)], ids=str)
@pytest.mark.parametrize("shift", [4, 8, 12])
def test_scales_at_any_four_bytes(lib, shape, shift):
    lens, Hq, Hkv, D, page = shape
    s = make(13, lens, Hq, Hkv, D, page)
    want = decode(lib, s)
    for at in (2, 3):
        t = s["pool"][at]
        room = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda")
        room[shift: shift + t.numel()] = t.flatten()
        s["pool"][at] = room[shift: shift + t.numel()].view(t.shape)
    out, lse, err = decode(lib, s)
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    s["pool"][2] = torch.zeros(s["pool"][2].numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(s["pool"][2].shape)
    with pytest.raises(lib.PagedKVError, match="invalid"):
        decode(lib, s)


def test_shared_pages(lib):
    """Two requests that list the same pages."""
    s = make(12, (128, 100), 8, 2, 128, 16)
    s["pages"][8: 8 + 4] = s["pages"][:4]
    s["rows"][1][:64] = s["rows"][0][:64]
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_pool_past_32_bits(lib):
    """Slots whose byte offsets pass 4 GB, for the append, the decode (boxes and rows), the read-back and a page's copy."""
    first = 530_000  # pages of 8 KB
    pool = [torch.zeros(first + 41, 16, 8, n, dtype=torch.uint8, device="cuda") for n in (64, 64, 8, 8)]
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(300, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(1, 32, 128, generator=gen).to(torch.bfloat16).cuda()
    slots = first * 16 + torch.randperm(320, generator=gen)[:300].cuda()
    scales = dict(k_global=KG, v_global=VG)
    lib.kv_append_fp4(*pool, k, v, slots, **scales)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    flat = [x.view(-1, 1, *x.shape[2:]) for x in pool]
    out, lse = lib.paged_decode_fp4(q, *flat, i32([0, 300]), slots.int(), i32([300]), 0.1, **scales)
    kd, vd = (cache4.values(*cache4.quantise(oracle.as_f64(x), g), g) for x, g in ((k, KG), (v, VG)))
    qd, o, l = oracle.as_f64(q)[0], oracle.as_f64(out)[0], oracle.as_f64(lse)[0]
    for h in range(8):
        a = attend(qd[4 * h: 4 * h + 4], kd[:, h], vd[:, h], 0.1)
        extra = 2.0 ** -32 * a[4].max(-1)[:, None] * np.abs(vd[:, h]).sum(0)
        check(o[4 * h: 4 * h + 4], l[4 * h: 4 * h + 4], a, 300, F16, f"head {h}", extra)
    ko, vo = (torch.zeros(320, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = i32(list(range(first, first + 20)))
    lib.paged_gather_fp4(*pool, i32([0, 20]), pages, i32([320]), i32([0, 320]), ko, vo, **scales)
    for got, want in ((ko, kd), (vo, vd)):
        assert torch.equal(got[slots - first * 16].cpu(), torch.tensor(want).float().to(torch.bfloat16))
    # the same rows as pages of 16, in page order, and as copies of those pages
    o16, l16 = lib.paged_decode_fp4(q, *pool, i32([0, 20]), pages, i32([320]), 0.1, **scales)
    small = [x[first:].contiguous() for x in pool]
    o2, l2 = lib.paged_decode_fp4(q, *small, i32([0, 20]), pages - first, i32([320]), 0.1, **scales)
    assert torch.equal(o16, o2) and torch.equal(l16, l2)
    lib.copy_pages(pool, pages, pages + 20)
    o3, l3 = lib.paged_decode_fp4(q, *pool, i32([0, 20]), pages + 20, i32([320]), 0.1, **scales)
    assert torch.equal(o16, o3) and torch.equal(l16, l3)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (8, 2), (14, 2), (9, 3), (24, 4), (64, 4), (30, 6), (12, 12), (40, 10)])
def test_head_dim_64_with_heads_in_pairs_and_single(lib, Hq, Hkv, page):
    """An even number of KV heads to a CTA lies in pairs in a box's rows; steps with half and all of their positions."""
    s = make(Hq + page, (200, 64, 31, 97, 1), Hq, Hkv, 64, page)
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (7, 1, 64), (32, 8, 128)])
@pytest.mark.parametrize("B", [1, 9, 10, 32, 33])
def test_merges_of_few_and_of_many_units(lib, B, Hq, Hkv, D):
    """One warp and eight for a head's partials; the unit's CTAs worked out by the merge (32 requests) and read (33)."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(1, 3000 // B + 40, B)]
    lens[B // 2] = 6000 // B + 700
    if B > 2:
        lens[0] = 0  # reported; its neighbours' shares do not move
    s = make(B, lens, Hq, Hkv, D, 16, "any")
    out, lse, err = decode(lib, s)
    assert err == (lib.DEVERR_LENGTH if B > 2 else 0)
    if B > 2:
        assert not out[0].any() and (lse[0] == float("-inf")).all()
    keep = [b for b in range(B) if lens[b]]
    s.update(q=s["q"][keep], lens=[lens[b] for b in keep], rows=[s["rows"][b] for b in keep])
    verify(s, out[keep], lse[keep])


def test_shares_whose_weights_are_all_0(lib):
    """Scores far below the others': the CTAs that hold them leave weights of 0, not NaN, to the merge."""
    s = make(12, (9000,), 8, 1, 128, 16)
    far = np.arange(9000) < 8900
    s["scale"][0][s["rows"][0][far]] = 0x7E  # 448
    s["codes"][0][s["rows"][0][far]] = 0xFF  # -6
    s["pool"][0].copy_(torch.tensor(s["codes"][0]).view(s["pool"][0].shape))
    s["pool"][2].copy_(torch.tensor(s["scale"][0]).view(s["pool"][2].shape))
    s["q"] = s["q"].abs() + 1
    out, lse, err = decode(lib, s)
    assert err == 0
    verify(s, out, lse)
