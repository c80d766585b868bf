"""The 4-bit cache's write and read-back against the fp64 oracle.  Without a rotation every byte is known and nothing has
a tolerance.  A rotated K is known up to the rotation's fp32 arithmetic, 2^-22 (|x_a| + |x_b|), so its scale may
be off by half a step (2^-4 of it, or 2^-10) from that, and its codes by half of theirs."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache4, cache8
from _gpu_helpers import bits_equal
from test_gpu_rotary_append import _pair_size, _table

pytestmark = pytest.mark.gpu


def empty(num_pages, page, Hkv, D, byte=0x55, scale=0x3A):
    p = [torch.full((num_pages, page, Hkv, D // 2), byte, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return p + [torch.full((num_pages, page, Hkv, D // 16), scale, dtype=torch.uint8, device="cuda") for _ in range(2)]


def rows(seed, T, Hkv, D):
    """Rows of many sizes, with zero blocks, blocks of one value, values on ties of the codes and of the scales, and values past
    both ends of what the cache can hold."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, Hkv, D // 16, 16)) * 2.0 ** rng.integers(-6, 7, (T, Hkv, D // 16, 1))
    flat = x.reshape(-1, 16)
    for i in range(0, len(flat), 11):
        flat[i] = 0.0
    for i in range(1, len(flat), 11):
        flat[i, 1:] = 0.0
    ties = np.array([6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    for i in range(2, len(flat), 11):  # every mantissa of a scale
        flat[i] = ties * (1 + i % 8 / 8) * 2.0 ** (i % 9 - 4)
    for i in range(3, len(flat), 11):  # largest values whose sixth is a tie between two scales
        flat[i] = rng.uniform(-1, 1, 16)
        flat[i, 5] = 6 * (1 + (2 * (i % 8) + 1) / 16)
    for i in range(4, len(flat), 11):
        flat[i] *= 2.0 ** 40
    for i in range(5, len(flat), 11):
        flat[i] *= 2.0 ** -30
    return torch.tensor(x.reshape(T, Hkv, D), dtype=torch.float32).to(torch.bfloat16)


@pytest.mark.parametrize("as_bytes", [True, False])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 64, 1), (40, 8, 128, 16), (333, 3, 128, 24), (50, 2, 64, 16),
                                          (29, 5, 16, 3), (31, 2, 80, 16), (17, 1, 256, 64), (2000, 8, 128, 1)])
def test_append(lib, T, Hkv, D, page, as_bytes):
    k, v = rows(T, T, Hkv, D), rows(T + 1, T, Hkv, D)
    kg, vg = (1.0, 0.5) if as_bytes else (0.0113, 1.7)
    num_pages = T * 2 // page + 2
    slots = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(T))[:T]
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    pool = empty(num_pages, page, Hkv, D)
    want = [t.cpu().numpy().reshape(-1, *t.shape[2:]) for t in pool]
    given = pool if as_bytes else pool[:2] + [t.view(torch.float8_e4m3fn) for t in pool[2:]]
    lib.kv_append_fp4(*given, k.cuda(), v.cuda(), slots.cuda(), k_global=kg, v_global=vg)
    live = (slots >= 0).numpy()
    to = slots.numpy()[live]
    for x, at, g in ((k, 0, kg), (v, 1, vg)):
        codes, scale = cache4.quantise(oracle.as_f64(x), g)
        want[at][to], want[2 + at][to] = codes[live], scale[live]
    for i, (t, w) in enumerate(zip(pool, want)):
        np.testing.assert_array_equal(t.cpu().numpy().reshape(w.shape), w, err_msg=str(i))


@pytest.mark.parametrize("g", [2.0 ** -64, 2.0 ** 64, 3e-10])
def test_append_with_extreme_cache_scales(lib, g):
    x = torch.cat([rows(3, 20, 2, 64).float() * s for s in (1.0, g, g * 1e20 if g < 1 else g * 1e-8)]).to(torch.bfloat16)
    pool = empty(4, 16, 2, 64)
    lib.kv_append_fp4(*pool, x.cuda(), x.cuda(), torch.arange(60).cuda(), k_global=g, v_global=g)
    codes, scale = cache4.quantise(oracle.as_f64(x), g)
    np.testing.assert_array_equal(pool[2].cpu().numpy().reshape(64, 2, 4)[:60], scale)
    np.testing.assert_array_equal(pool[1].cpu().numpy().reshape(64, 2, 32)[:60], codes)


def test_append_of_infinities_and_nans(lib):
    """They make their block NaN and leave the others alone."""
    k = rows(5, 6, 2, 64)
    v = k.clone()
    v[0, 0, 3], v[1, 1, 0], v[2, 0, 63], v[3, 1, :] = float("inf"), float("nan"), float("-inf"), float("nan")
    pool = empty(1, 8, 2, 64)
    lib.kv_append_fp4(*pool, k.cuda(), v.cuda(), torch.arange(6).cuda())
    codes, scale = cache4.quantise(oracle.as_f64(v), 1.0)
    assert (scale == 0x7F).sum() == 1 + 1 + 1 + 4
    np.testing.assert_array_equal(pool[1].cpu().numpy().reshape(8, 2, 32)[:6], codes)
    np.testing.assert_array_equal(pool[3].cpu().numpy().reshape(8, 2, 4)[:6], scale)


def test_append_reports_a_slot_past_the_pool(lib):
    k = rows(6, 3, 2, 64)
    pool = empty(2, 4, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kv_append_fp4(*pool, k.cuda(), k.cuda(), torch.tensor([8, 1, -5]).cuda(), err_word=err)
    assert int(err) == lib.DEVERR_SLOT_OOB
    changed = (pool[0] != 0x55).flatten(2).any(-1).flatten().cpu()
    assert torch.nonzero(changed).flatten().tolist() == [1]


ROTATIONS = [
    # T, Hkv, Hq, D, R, interleaved, page, pad
    (1, 1, 1, 64, 64, False, 16, 0),
    (5, 2, 14, 64, 64, True, 16, 1),
    (131, 8, 32, 128, 128, False, 16, 17),
    (77, 3, 6, 128, 32, False, 24, 0),
    (64, 4, 4, 128, 64, True, 1, 0),
    (33, 2, 4, 80, 48, False, 8, 3),   # a half of an odd number of chunks
    (33, 2, 4, 80, 20, False, 8, 3),
    (33, 2, 4, 80, 22, True, 8, 3),
    (40, 1, 3, 16, 16, False, 4, 0),
    (21, 2, 2, 256, 96, False, 16, 0),
    (21, 2, 0, 256, 256, False, 16, 2),
    (300, 8, 16, 128, 8, True, 16, 0),
]


@pytest.mark.parametrize("T,Hkv,Hq,D,R,interleaved,page,pad", ROTATIONS)
@pytest.mark.parametrize("in_place", [True, False])
def test_rotary_append(lib, T, Hkv, Hq, D, R, interleaved, page, pad, in_place):
    gen = torch.Generator().manual_seed(T + R)
    rn = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)  # noqa: E731
    k, v, q = rn(T, Hkv, D) * 3, rn(T, Hkv, D), rn(T, Hq, D) if Hq else None
    pos = torch.randint(0, 4096, (T,), generator=gen, dtype=torch.int32)
    table = _table(R)
    num_pages = T * 5 // 4 // page + 2
    slots = torch.randperm(num_pages * page, generator=gen)[:T]
    slots[torch.randperm(T, generator=gen)[:pad]] = -1
    pool = empty(num_pages, page, Hkv, D)
    before = [t.clone() for t in pool]
    kg, vg = 0.0113, 0.00235
    qd = q.cuda() if Hq else None
    q_out = None if in_place or not Hq else torch.empty_like(qd)
    lib.rotary_kv_append_fp4(*pool, k.cuda(), v.cuda(), slots.cuda(), pos.cuda(), table.cuda(), q=qd, q_out=q_out,
                             interleaved=interleaved, k_global=kg, v_global=vg)
    live = (slots >= 0).numpy()
    to = slots.numpy()[live]
    got = [t.cpu().numpy().reshape(-1, *t.shape[2:]) for t in pool]
    # V, and every slot that is not written
    codes, scale = cache4.quantise(oracle.as_f64(v), vg)
    np.testing.assert_array_equal(got[1][to], codes[live])
    np.testing.assert_array_equal(got[3][to], scale[live])
    rest = np.ones(num_pages * page, dtype=bool)
    rest[to] = False
    for t, w in zip(got, before):
        np.testing.assert_array_equal(t[rest], w.cpu().numpy().reshape(t.shape)[rest])
    # K
    x = cache8.rotate(k, table, pos, interleaved)[live]
    eps = 2.0 ** -22 * _pair_size(k, R, interleaved)[live]
    g = float(np.float32(kg))
    blocks, off = x.reshape(*x.shape[:-1], -1, 16), eps.reshape(*x.shape[:-1], -1, 16)
    s = cache8.e4m3_values(got[2][to])
    exact = np.abs(blocks).max(-1) / (6 * g)
    assert np.all(np.abs(s - exact) <= np.maximum(2.0 ** -4 * exact, 2.0 ** -10) * (1 + 2.0 ** -20) + off.max(-1) / (6 * g))
    y = np.abs(blocks) / (s * g)[..., None]
    c = cache4.e2m1_values(cache4.unpack(got[0][to])).reshape(blocks.shape)
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
    slack = off / (s * g)[..., None] + 2.0 ** -20
    assert np.all((np.abs(c) == 6) | (np.abs(np.abs(c) - y) <= half + slack))
    assert np.all((np.abs(c) != 6) | (y >= 5 - slack))
    assert np.all((c == 0) | (np.sign(c) == np.sign(blocks)) | (y <= 0.25 + slack))
    if Hq:
        turned = cache8.rotate(q, table, pos, interleaved)
        out = oracle.as_f64(q_out if q_out is not None else qd)
        assert np.all(np.abs(out - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -21 * (_pair_size(q, R, interleaved)))


GATHERS = [
    # lens, gaps behind each request's rows, Hkv, D, page
    ([1], [0], 1, 64, 16),
    ([0, 5, 0, 0, 33, 16], [0, 3, 0, 7, 0, 16], 8, 128, 16),
    ([100, 1, 64], [0, 0, 0], 3, 128, 1),
    ([17, 18, 19, 500], [15, 14, 13, 0], 2, 64, 24),
    ([40, 7], [2, 0], 5, 48, 8),
    ([3] * 300, [1] * 300, 4, 64, 2),
]


@pytest.mark.parametrize("g", [0.25, 0.0113])
@pytest.mark.parametrize("lens,gaps,Hkv,D,page", GATHERS, ids=lambda x: str(x)[:24])
def test_gather(lib, lens, gaps, Hkv, D, page, g):
    rng = np.random.default_rng(sum(lens))
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 3
    perm = rng.permutation(num_pages)[: sum(need)]
    codes = rng.integers(0, 256, (2, num_pages, page, Hkv, D // 2)).astype(np.uint8)
    scale = rng.integers(0, 127, (2, num_pages, page, Hkv, D // 16)).astype(np.uint8)  # every scale but NaN
    indptr = np.concatenate([[0], np.cumsum(need)])
    starts = 2 + np.concatenate([[0], np.cumsum(np.array(lens) + np.array(gaps))])
    N = int(starts[-1]) + 5
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    ko = torch.full((N, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, -9.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_gather_fp4(*[torch.tensor(c).cuda() for c in codes], *[torch.tensor(x).cuda() for x in scale],
                         i32(indptr), i32(perm), i32(lens), i32(starts), ko, vo, k_global=g, v_global=2 * g, err_word=err)
    assert int(err) == 0
    for at, (out, fill) in enumerate(((ko, 9.0), (vo, -9.0))):
        want = torch.full((N, Hkv, D), fill, dtype=torch.bfloat16)
        held = cache4.values(codes[at], scale[at], g * (1 + at))
        for b, n in enumerate(lens):
            for j in range(n):
                # the kernel's fp32 product rounds the exact one once, as .float() does here
                want[starts[b] + j] = torch.tensor(held[perm[indptr[b] + j // page], j % page]).float().to(torch.bfloat16)
        assert bits_equal(out, want)


def test_append_then_read_back(lib):
    """With a power of two as the cache's scale the read-back has no rounding of its own."""
    T, Hkv, D, page = 100, 4, 128, 16
    k, v = rows(1, T, Hkv, D), rows(2, T, Hkv, D)
    pool = empty(8, page, Hkv, D)
    slots = torch.randperm(8 * page, generator=torch.Generator().manual_seed(0))[:T]
    lib.kv_append_fp4(*pool, k.cuda(), v.cuda(), slots.cuda(), k_global=0.125, v_global=2.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ko, vo = (torch.empty(8 * page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.paged_gather_fp4(*pool, i32([0, 8]), i32(list(range(8))), i32([8 * page]), i32([0, 8 * page]), ko, vo,
                         k_global=0.125, v_global=2.0)
    for x, out, g in ((k, ko, 0.125), (v, vo, 2.0)):
        want = cache4.values(*cache4.quantise(oracle.as_f64(x), g), g)
        assert np.array_equal(oracle.as_f64(out)[slots.numpy()], want)


def test_gather_reports_what_it_skips(lib):
    pool = empty(4, 4, 2, 64, byte=0x22, scale=0x38)  # all values 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731

    def run(indptr, pages, lens, starts, rows=32):
        ko, vo = (torch.zeros(rows, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.paged_gather_fp4(*pool, i32(indptr), i32(pages), i32(lens), i32(starts), ko, vo, err_word=err)
        assert torch.equal(ko, vo)
        return int(err), torch.nonzero(ko[:, 0, 0]).flatten().tolist()

    assert run([0, 1, 2], [0, 1], [4, 3], [0, 4, 8]) == (0, [0, 1, 2, 3, 4, 5, 6])
    assert run([0, 1, 2], [0, 9], [4, 3], [0, 4, 8]) == (lib.DEVERR_PAGE_OOB, [0, 1, 2, 3])
    assert run([0, 1, 2], [0, -1], [4, 3], [0, 4, 8]) == (lib.DEVERR_PAGE_OOB, [0, 1, 2, 3])
    assert run([0, 1, 2], [0, 1], [6, 3], [0, 6, 9]) == (lib.DEVERR_LENGTH, [0, 1, 2, 3, 6, 7, 8])
    assert run([0, 1, 2], [0, 1], [4, 3], [0, 30, 33]) == (lib.DEVERR_ROW_OOB, [0, 1, 2, 3, 30, 31])


@pytest.mark.parametrize("k_off,v_off", [(8, 0), (0, 8), (8, 24), (16, 32)])
def test_gather_into_rows_that_begin_at_16_bytes(lib, k_off, v_off):
    """Any 16-byte aligned place for the results will do, in a tensor of more rows' memory."""
    N, Hkv, D, page = 50, 2, 64, 16
    rng = np.random.default_rng(8)
    codes = rng.integers(0, 256, (2, 4, page, Hkv, D // 2)).astype(np.uint8)
    scale = rng.integers(0, 127, (2, 4, page, Hkv, D // 16)).astype(np.uint8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    flat = [torch.full((N * Hkv * D + 64,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ko, vo = (f[o: o + N * Hkv * D].view(N, Hkv, D) for f, o in zip(flat, (k_off, v_off)))
    lib.paged_gather_fp4(*[torch.tensor(c).cuda() for c in codes], *[torch.tensor(x).cuda() for x in scale], i32([0, 4]),
                         i32([2, 0, 3, 1]), i32([N]), i32([0, N]), ko, vo, k_global=0.25, v_global=0.5)
    for at, (f, out, off) in enumerate(((flat[0], ko, k_off), (flat[1], vo, v_off))):
        held = cache4.values(codes[at], scale[at], 0.25 * (1 + at))[[2, 0, 3, 1]].reshape(-1, Hkv, D)[:N]
        assert bits_equal(out, torch.tensor(held).float().to(torch.bfloat16))
        assert (f[:off] == 7.0).all() and (f[off + N * Hkv * D:] == 7.0).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_gather_of_empty_prefixes_alone(lib, bits):
    """A batch in which nobody has a page: an empty list of pages, and rows that stay what they were."""
    pool = empty(2, 16, 2, 64) if bits == 4 else [torch.zeros(2, 16, 2, 64, dtype=torch.float8_e4m3fn, device="cuda")] * 2 + [
        torch.ones(2, 16, 2, device="cuda")] * 2
    gather = lib.paged_gather_fp4 if bits == 4 else lib.paged_gather_fp8
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ko = torch.full((6, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vo, err = ko.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    gather(*pool, i32(0, 0, 0), i32(), i32(0, 0), i32(0, 3, 6), ko, vo, err_word=err)
    assert int(err) == 0
    gather(*pool, i32(0, 0, 0), i32(), i32(0, 2), i32(0, 3, 6), ko, vo, err_word=err)
    assert int(err) == lib.DEVERR_LENGTH
    gather(*pool, i32(0, 1, 1), i32(), i32(2, 0), i32(0, 3, 6), ko, vo, err_word=err)  # a list that is not there
    assert int(err) == lib.DEVERR_LENGTH
    assert (ko == 3.0).all() and (vo == 3.0).all()
