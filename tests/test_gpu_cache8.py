"""The 8-bit cache's write and read-back against the fp64 oracle: every byte is known, so nothing
here has a tolerance."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from _gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu


def _empty(num_pages, page, Hkv, D, byte=0x55, scale=3.0):
    p = [torch.full((num_pages, page, Hkv, D), byte, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return p + [torch.full((num_pages, page, Hkv), scale, device="cuda") for _ in range(2)]


def _rows(seed, T, Hkv, D):
    """Rows of many sizes, with zero rows, denormal rows, rows of one value and values on ties."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, Hkv, D)) * 2.0 ** rng.integers(-20, 20, (T, Hkv, 1))
    for i in range(0, T, 7):
        x[i, 0] = 0.0
    for i in range(1, T, 7):
        x[i, -1] = rng.standard_normal(D) * 2.0 ** -128
    for i in range(2, T, 7):
        x[i, 0, 1:] = 0.0
    for i in range(3, T, 7):  # 448 sets the scale to 1, 17 and 19 are ties of e4m3
        x[i, -1] = np.resize([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, -(2.0 ** -9), 3 * 2.0 ** -10, -0.0], D)
    for i in range(4, T, 7):
        x[i, 0] = np.resize([3.3e38, -1.0, 2.0 ** 100], D)
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


@pytest.mark.parametrize("as_bytes", [True, False])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 64, 1), (40, 8, 128, 16), (333, 3, 128, 24), (50, 2, 64, 16),
                                          (29, 5, 8, 3), (31, 2, 80, 16), (17, 1, 256, 64), (2000, 8, 128, 1)])
def test_append(lib, T, Hkv, D, page, as_bytes):
    k, v = _rows(T, T, Hkv, D), _rows(T + 1, T, Hkv, D)
    num_pages = T * 2 // page + 2
    slots = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(T))[:T]
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    pool = _empty(num_pages, page, Hkv, D)
    want = [t.cpu().numpy().reshape(-1, *t.shape[2:]) for t in pool]
    given = [t.view(torch.float8_e4m3fn) for t in pool[:2]] + pool[2:] if not as_bytes else pool
    lib.kv_append_fp8(*given, k.cuda(), v.cuda(), slots.cuda())
    live = (slots >= 0).numpy()
    to = slots.numpy()[live]
    for x, at, scale_at in ((k, 0, 2), (v, 1, 3)):
        codes, scale = cache8.quantise(oracle.as_f64(x))
        want[at][to], want[scale_at][to] = codes[live], scale[live]
    for t, w in zip(pool, want):
        np.testing.assert_array_equal(t.cpu().numpy().reshape(w.shape), w)


def test_append_of_infinities_and_nans(lib):
    """They are stored as NaN and leave the row's scale and its other values alone."""
    k = _rows(5, 6, 2, 64)
    v = k.clone()
    v[0, 0, 3], v[1, 1, 0], v[2, 0, 63], v[3, 1, :] = float("inf"), float("nan"), float("-inf"), float("nan")
    pool = _empty(1, 8, 2, 64)
    lib.kv_append_fp8(*pool, k.cuda(), v.cuda(), torch.arange(6).cuda())
    codes, scale = cache8.quantise(oracle.as_f64(v))
    got = pool[1].cpu().numpy().reshape(8, 2, 64)[:6]
    np.testing.assert_array_equal(cache8.e4m3_values(got), cache8.e4m3_values(codes))
    np.testing.assert_array_equal(pool[3].cpu().numpy().reshape(8, 2)[:6], scale)


def test_append_reports_a_slot_past_the_pool(lib):
    k = _rows(6, 3, 2, 64)
    pool = _empty(2, 4, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kv_append_fp8(*pool, k.cuda(), k.cuda(), torch.tensor([8, 1, -5]).cuda(), err_word=err)
    assert int(err) == lib.DEVERR_SLOT_OOB
    changed = (pool[0] != 0x55).flatten(2).any(-1).flatten().cpu()
    assert torch.nonzero(changed).flatten().tolist() == [1]


GATHERS = [
    # lens, gaps behind each request's rows, Hkv, D, page
    ([1], [0], 1, 64, 16),
    ([0, 5, 0, 0, 33, 16], [0, 3, 0, 7, 0, 16], 8, 128, 16),
    ([100, 1, 64], [0, 0, 0], 3, 128, 1),
    ([17, 18, 19, 500], [15, 14, 13, 0], 2, 64, 24),
    ([40, 7], [2, 0], 5, 24, 8),
    ([3] * 300, [1] * 300, 4, 64, 2),
]


@pytest.mark.parametrize("lens,gaps,Hkv,D,page", GATHERS, ids=lambda x: str(x)[:24])
def test_gather(lib, lens, gaps, Hkv, D, page):
    rng = np.random.default_rng(sum(lens))
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 3
    perm = rng.permutation(num_pages)[: sum(need)]
    # every byte but the NaN codes, and scales that are not powers of two for half of the rows
    codes = rng.integers(0, 254, (2, num_pages, page, Hkv, D)).astype(np.uint8)
    codes = np.where((codes & 0x7F) == 0x7F, 0, codes).astype(np.uint8)
    scale = 2.0 ** rng.integers(-20, 20, (2, num_pages, page, Hkv))
    scale[:, ::2] *= 1 + rng.random((2, (num_pages + 1) // 2, page, Hkv)).astype(np.float32)
    scale = scale.astype(np.float32)
    indptr = np.concatenate([[0], np.cumsum(need)])
    starts = 2 + np.concatenate([[0], np.cumsum(np.array(lens) + np.array(gaps))])
    N = int(starts[-1]) + 5
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    ko = torch.full((N, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, -9.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_gather_fp8(*[torch.tensor(c).cuda() for c in codes], *[torch.tensor(x).cuda() for x in scale],
                         i32(indptr), i32(perm), i32(lens), i32(starts), ko, vo, err_word=err)
    assert int(err) == 0
    for at, (out, fill) in enumerate(((ko, 9.0), (vo, -9.0))):
        want = torch.full((N, Hkv, D), fill, dtype=torch.bfloat16)
        for b, n in enumerate(lens):
            for j in range(n):
                pg, r = perm[indptr[b] + j // page], j % page
                x = cache8.e4m3_values(codes[at, pg, r]) * scale[at, pg, r].astype(np.float64)[:, None]
                # the kernel's fp32 product rounds the exact one once, as .float() does here
                want[starts[b] + j] = torch.tensor(x).float().to(torch.bfloat16)
        assert bits_equal(out, want)


def test_append_then_read_back_is_exact(lib):
    """bf16(x8 * 2^k) has no rounding of its own: reading back gives the values the bytes stand for."""
    T, Hkv, D, page = 100, 4, 128, 16
    k, v = _rows(1, T, Hkv, D), _rows(2, T, Hkv, D)
    pool = _empty(8, page, Hkv, D)
    slots = torch.randperm(8 * page, generator=torch.Generator().manual_seed(0))[:T]
    lib.kv_append_fp8(*pool, k.cuda(), v.cuda(), slots.cuda())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ko, vo = (torch.empty(8 * page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.paged_gather_fp8(*pool, i32([0, 8]), i32(list(range(8))), i32([8 * page]), i32([0, 8 * page]), ko, vo)
    for x, out in ((k, ko), (v, vo)):
        codes, scale = cache8.quantise(oracle.as_f64(x))
        want = torch.tensor(cache8.e4m3_values(codes) * scale[..., None]).float().to(torch.bfloat16)
        assert torch.equal(want.double(), torch.tensor(cache8.e4m3_values(codes) * scale[..., None]))
        assert torch.equal(out.cpu()[slots].double(), want.double())


def test_gather_reports_what_it_skips(lib):
    pool = _empty(4, 4, 2, 64, byte=0x38, scale=1.0)  # all values 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731

    def run(indptr, pages, lens, starts, rows=32):
        ko, vo = (torch.zeros(rows, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.paged_gather_fp8(*pool, i32(indptr), i32(pages), i32(lens), i32(starts), ko, vo, err_word=err)
        assert torch.equal(ko, vo)
        return int(err), torch.nonzero(ko[:, 0, 0]).flatten().tolist()

    assert run([0, 1, 2], [0, 1], [4, 3], [0, 4, 8]) == (0, [0, 1, 2, 3, 4, 5, 6])
    assert run([0, 1, 2], [0, 9], [4, 3], [0, 4, 8]) == (lib.DEVERR_PAGE_OOB, [0, 1, 2, 3])
    assert run([0, 1, 2], [0, -1], [4, 3], [0, 4, 8]) == (lib.DEVERR_PAGE_OOB, [0, 1, 2, 3])
    assert run([0, 1, 2], [0, 1], [6, 3], [0, 6, 9]) == (lib.DEVERR_LENGTH, [0, 1, 2, 3, 6, 7, 8])
    assert run([0, 2, 3], [0, 1, 2], [6, 3], [0, 4, 8]) == (lib.DEVERR_LENGTH, [0, 1, 2, 3, 4, 5, 6])
    assert run([0, 1, 2], [0, 1], [4, 3], [0, 30, 33]) == (lib.DEVERR_ROW_OOB, [0, 1, 2, 3, 30, 31])
