"""Copies of pages and the compaction of accepted tokens: bytes move, so nothing here has a tolerance."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def cache(seed, kind, num_pages, page, Hkv, D, layers=1):
    """The tensors of all layers' caches, filled with random bytes."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    head = (num_pages, page, Hkv)
    shapes = {"bf16": [((D,), torch.bfloat16)] * 2,
              "8 bits": [((D,), torch.float8_e4m3fn)] * 2 + [((), torch.float32)] * 2,
              "4 bits": [((D // 2,), torch.uint8)] * 2 + [((D // 16,), torch.float8_e4m3fn)] * 2}[kind]
    out = []
    for _ in range(layers):
        for tail, dtype in shapes:
            n = torch.empty(0, dtype=dtype).element_size()
            raw = torch.randint(0, 256, (*head, *tail[:-1], (tail[-1] if tail else 1) * n), generator=gen, device="cuda",
                                dtype=torch.uint8)
            out.append(raw.view(dtype).view(*head, *tail))
    return out


def raw(t):
    """A tensor's bytes as [slots, bytes]."""
    return t.contiguous().view(t.shape[0] * t.shape[1], -1).view(torch.uint8).cpu().numpy()


def check(tensors, before, src_slots, dst_slots):
    """Every tensor is what it was with the rows src_slots (as they were) at dst_slots."""
    for i, (t, b) in enumerate(zip(tensors, before)):
        want = b.copy()
        want[dst_slots] = b[src_slots]
        np.testing.assert_array_equal(raw(t), want, err_msg=f"tensor {i}")


SHAPES = [
    # kind, page, Hkv, D, layers
    ("bf16", 16, 8, 128, 1),
    ("bf16", 1, 1, 8, 2),
    ("bf16", 24, 3, 72, 5),
    ("8 bits", 16, 8, 128, 1),
    ("8 bits", 1, 1, 24, 3),
    ("8 bits", 5, 7, 64, 9),
    ("4 bits", 16, 8, 128, 36),
    ("4 bits", 1, 1, 64, 4),
    ("4 bits", 3, 1, 16, 2),     # one byte of scales a slot
    ("4 bits", 8, 3, 32, 64),    # 256 tensors
    ("4 bits", 64, 16, 256, 2),
]


@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("kind,page,Hkv,D,layers", SHAPES)
@pytest.mark.parametrize("copies", [1, 13])
def test_copy_pages(lib, kind, page, Hkv, D, layers, copies, partial):
    rng = np.random.default_rng(copies + page)
    num_pages = 2 * copies + 3
    tensors = cache(1, kind, num_pages, page, Hkv, D, layers)
    before = [raw(t) for t in tensors]
    perm = rng.permutation(num_pages)
    dst = perm[:copies].copy()
    src = rng.choice(perm[copies:], copies)  # a page may be copied several times
    if copies > 1:
        dst[3] = -1  # padding
        src[4] = dst[4]  # onto itself
    rows = rng.integers(0, page + 1, copies) if partial else np.full(copies, page)
    err = torch.zeros(1, **I32)
    lib.copy_pages(tensors, i32(src), i32(dst), rows=i32(rows) if partial else None, err_word=err)
    assert int(err) == 0
    moves = [(s * page + r, d * page + r) for s, d, n in zip(src, dst, rows) if d >= 0 for r in range(n)]
    moves = np.array(moves, dtype=np.int64).reshape(-1, 2)
    check(tensors, before, moves[:, 0], moves[:, 1])


@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_tensors_at_any_place(lib, shift):
    """Views that do not begin at a multiple of 16 bytes, beside one that does."""
    def view(shape):
        n = int(np.prod(shape))
        return torch.randint(0, 256, (n + 16,), dtype=torch.uint8, device="cuda")[shift: shift + n].view(shape)

    tensors = [view((9, 4, 2, 64)), view((9, 4, 2, 4)), cache(8, "bf16", 9, 4, 2, 64)[0], view((9, 4, 33))]
    before = [raw(x) for x in tensors]
    lib.copy_pages(tensors, i32([0, 1]), i32([7, 8]), rows=i32([3, 4]))
    src, dst = [0, 1, 2, 4, 5, 6, 7], [28, 29, 30, 32, 33, 34, 35]
    check(tensors, before, src, dst)
    before = [raw(x) for x in tensors]
    lib.compact_accepted(tensors, i32([0, 3]), i32([2, 5, 3]), i32([2]), i32([0, 4]), i32([1, 3, 4, 9]))
    slot = lambda p: [2, 5, 3][p // 4] * 4 + p % 4  # noqa: E731
    check(tensors, before, [slot(p) for p in (3, 5, 6, 11)], [slot(p) for p in (2, 3, 4, 5)])


def test_copy_reports_what_it_skips(lib):
    def run(src, dst, rows=None):
        t = cache(2, "bf16", 6, 4, 2, 64)
        before = [raw(x) for x in t]
        err = torch.zeros(1, **I32)
        lib.copy_pages(t, i32(src), i32(dst), rows=None if rows is None else i32(rows), err_word=err)
        changed = [(raw(x) != b).reshape(6, 4, -1).any(-1) for x, b in zip(t, before)]
        assert np.array_equal(changed[0], changed[1])
        return int(err), np.argwhere(changed[0]).tolist()

    all_of = lambda p: [[p, r] for r in range(4)]  # noqa: E731
    assert run([0, 1], [2, 3]) == (0, all_of(2) + all_of(3))
    assert run([0, 6], [2, 3]) == (lib.DEVERR_PAGE_OOB, all_of(2))
    assert run([-1, 1], [2, 3]) == (lib.DEVERR_PAGE_OOB, all_of(3))
    assert run([0, 1], [6, 3]) == (lib.DEVERR_PAGE_OOB, all_of(3))
    assert run([6, 1], [-2, 3]) == (0, all_of(3))
    assert run([0, 1], [2, 3], [5, 2]) == (lib.DEVERR_LENGTH, [[3, 0], [3, 1]])
    assert run([0, 1], [2, 3], [-1, 0]) == (lib.DEVERR_LENGTH, [])


def trees(rng, B, nodes, page, prefix_most):
    """Page lists, prefixes and accepted nodes of B requests."""
    prefix = rng.integers(0, prefix_most + 1, B)
    need = -(-(prefix + nodes) // page)
    num_pages = int(need.sum()) + 3
    perm = rng.permutation(num_pages)[: need.sum()]
    indptr = np.concatenate([[0], np.cumsum(need)])
    accepted = [np.sort(rng.choice(nodes, rng.integers(0, nodes + 1), replace=False)) for _ in range(B)]
    src, dst = [], []
    for b, a in enumerate(accepted):
        slot = lambda pos: perm[indptr[b] + pos // page] * page + pos % page  # noqa: E731, B023
        for k, node in enumerate(a):
            src.append(slot(prefix[b] + node))
            dst.append(slot(prefix[b] + k))
    starts = np.concatenate([[0], np.cumsum([len(a) for a in accepted])])
    return dict(num_pages=num_pages, src=np.array(src, dtype=np.int64), dst=np.array(dst, dtype=np.int64),
                args=(i32(indptr), i32(perm), i32(prefix), i32(starts), i32(np.concatenate(accepted))))


@pytest.mark.parametrize("B,nodes", [(1, 1), (1, 8), (9, 16), (3, 64), (2, 300)])
@pytest.mark.parametrize("kind,page,Hkv,D,layers", SHAPES)
def test_compact_accepted(lib, kind, page, Hkv, D, layers, B, nodes):
    if nodes > 64 and layers > 4:
        pytest.skip("large")
    t = trees(np.random.default_rng(B + nodes), B, nodes, page, 40)
    tensors = cache(3, kind, t["num_pages"], page, Hkv, D, layers)
    before = [raw(x) for x in tensors]
    err = torch.zeros(1, **I32)
    lib.compact_accepted(tensors, *t["args"], err_word=err)
    assert int(err) == 0
    check(tensors, before, t["src"], t["dst"])


def test_compact_every_subset_of_a_small_tree(lib):
    """All 256 sets of accepted nodes of a tree of eight, chains of moves among them."""
    page, B = 4, 256
    indptr = 2 * np.arange(B + 1)
    perm = np.random.default_rng(0).permutation(2 * B)
    accepted = [[i for i in range(8) if s >> i & 1] for s in range(B)]
    tensors = cache(4, "8 bits", 2 * B, page, 2, 64)
    before = [raw(x) for x in tensors]
    starts = np.concatenate([[0], np.cumsum([len(a) for a in accepted])])
    lib.compact_accepted(tensors, i32(indptr), i32(perm), i32(np.zeros(B)), i32(starts), i32(sum(accepted, [])))
    slot = lambda b, p: perm[2 * b + p // page] * page + p % page  # noqa: E731
    src = [slot(b, n) for b, a in enumerate(accepted) for n in a]
    dst = [slot(b, k) for b, a in enumerate(accepted) for k in range(len(a))]
    check(tensors, before, src, dst)


def test_compact_reports_what_it_skips(lib):
    def run(accepted, starts=(0, 2, 4), prefix=(3, 2), pages=(0, 1, 2, 3)):
        """Two requests of two pages of four; which rows changed."""
        t = cache(5, "bf16", 6, 4, 2, 64)
        before = [raw(x) for x in t]
        err = torch.zeros(1, **I32)
        lib.compact_accepted(t, i32([0, 2, 4]), i32(pages), i32(prefix), i32(starts), i32(accepted), err_word=err)
        changed = [(raw(x) != b).any(-1) for x, b in zip(t, before)]
        assert np.array_equal(changed[0], changed[1])
        return int(err), np.flatnonzero(changed[0]).tolist()

    assert run([1, 2, 2, 4]) == (0, [3, 4, 10, 11])
    assert run([1, 1, 2, 4]) == (lib.DEVERR_LENGTH, [3, 10, 11])          # not ascending
    assert run([-1, 2, 2, 4]) == (lib.DEVERR_LENGTH, [4, 10, 11])
    assert run([1, 5, 2, 4]) == (lib.DEVERR_LENGTH, [3, 10, 11])          # position 8 of two pages of four
    assert run([1, 2 ** 31 - 1, 2, 4]) == (lib.DEVERR_LENGTH, [3, 10, 11])
    assert run([1, 2, 2, 4], prefix=(-1, 2)) == (lib.DEVERR_LENGTH, [10, 11])
    assert run([1, 2, 2, 4], starts=(0, 2, 5)) == (lib.DEVERR_ROW_OOB, [3, 4])
    assert run([1, 2, 2, 4], starts=(-1, 2, 4)) == (lib.DEVERR_ROW_OOB, [10, 11])
    assert run([1, 2, 2, 4], pages=(0, 6, 2, 3)) == (lib.DEVERR_PAGE_OOB, [10, 11])
    assert run([0, 1, 0, 1]) == (0, [])                                   # in their places already


def test_neither_touches_anything_when_there_is_nothing_to_do(lib):
    t = cache(6, "4 bits", 4, 8, 2, 64)
    before = [raw(x) for x in t]
    none = torch.zeros(0, **I32)
    lib.copy_pages(t, none, none)
    lib.compact_accepted(t, i32([0]), none, none, i32([0]), none)
    lib.compact_accepted(t, i32([0, 1]), i32([2]), i32([3]), i32([0, 0]), none)
    check(t, before, [], [])


def test_binding_refusals_on_the_device(lib):
    t = cache(7, "bf16", 4, 8, 2, 64)
    one = i32([1])
    with pytest.raises(ValueError, match="at least one"):
        lib.copy_pages([], one, one)
    with pytest.raises(ValueError, match="contiguous"):
        lib.copy_pages([t[0][:, :, :1]], one, one)
    with pytest.raises(ValueError, match="num_pages"):
        lib.copy_pages([t[0], t[1][:3]], one, one)
    with pytest.raises(ValueError, match="entries"):
        lib.copy_pages(t, one, i32([1, 2]))
    with pytest.raises(ValueError, match="entries"):
        lib.copy_pages(t, one, one, rows=i32([1, 2]))
    with pytest.raises(TypeError, match="int32"):
        lib.copy_pages(t, one.long(), one)
    with pytest.raises(lib.PagedKVError, match="unsupported"):
        lib.copy_pages([t[0]] * 257, one, one)
    with pytest.raises(ValueError, match="accepted_indptr"):
        lib.compact_accepted(t, i32([0, 1]), one, one, one, one)
    with pytest.raises(ValueError, match="kv_indptr"):
        lib.compact_accepted(t, one, one, one, i32([0, 1]), one)
