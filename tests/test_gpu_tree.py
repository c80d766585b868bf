"""Attention of drafted trees over a paged cache against 64-bit attention with the same mask."""

import math

import numpy as np
import pytest
import torch

import oracle
from _attention64 import attend, check

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # half a step: the weights of the second product are rounded to bf16


def tree_rows(rng, n, kind):
    """Visibility of n drafted tokens, bool [n, n]."""
    if kind == "chain":
        return np.tril(np.ones((n, n), dtype=bool))
    if kind == "random":  # any set, empty rows and rows that do not see themselves among them
        seen = rng.random((n, n)) < 0.3
        seen[rng.random(n) < 0.2] = False
        return seen
    if kind == "none":
        return np.zeros((n, n), dtype=bool)
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        p = int(rng.integers(max(0, i - 6), i)) if i and rng.random() < 0.9 else -1
        seen[i] = seen[p] if p >= 0 else False
        seen[i, i] = True
    return seen


def words_of(seen, words):
    """Mask rows of a request, int32 [n, words]."""
    n = seen.shape[0]
    bits = np.zeros((n, 32 * words), dtype=np.uint64)
    bits[:, :n] = seen
    w = (bits.reshape(n, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def make(seed, prefix, nodes, Hq, Hkv, D, page, kind="tree", extra_words=0, v_poison=True):
    """A step: pool slots that no request owns hold NaN, as do K and V of drafted tokens no row sees."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    lens = [p + n for p, n in zip(prefix, nodes)]
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 3
    perm = rng.permutation(num_pages)[: sum(need)]
    indptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    pools = [torch.full((num_pages * page, Hkv, D), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
    qo = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    words = -(-max(max(nodes), 1) // 32) + extra_words
    rows, seen, mask = [], [], []
    for b, n in enumerate(lens):
        j = np.arange(n)
        slot = torch.tensor(perm[indptr[b] + j // page].astype(np.int64) * page + j % page)
        rows.append(slot)
        s = tree_rows(rng, nodes[b], kind)
        seen.append(s)
        mask.append(words_of(s, words))
        for p in pools:
            p[slot] = torch.randn(n, Hkv, D, generator=gen).to(torch.bfloat16)
            if v_poison:
                p[slot[prefix[b]:][~torch.tensor(s.any(0))]] = float("nan")
    mask = torch.tensor(np.concatenate(mask)).cuda()
    if extra_words:  # bits of tokens that do not exist
        mask[:, -extra_words:] = -1
    q = torch.randn(int(qo[-1]), Hq, D, generator=gen).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    return dict(q=q.cuda(), k=pools[0].view(num_pages, page, Hkv, D).cuda(), v=pools[1].view(num_pages, page, Hkv, D).cuda(),
                qo=i32(qo), indptr=i32(indptr), pages=i32(perm), prefix=i32(prefix), mask=mask, most=max(max(nodes), 1),
                sm=1 / math.sqrt(D), rows=rows, seen=seen, host=(prefix, nodes, qo, Hq, Hkv))


def call(lib, s, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.paged_tree_attention(s["q"], s["k"], s["v"], s["qo"], s["indptr"], s["pages"], s["prefix"], s["mask"],
                                        s["most"], s["sm"], err_word=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


def verify(s, out, lse, requests=None):
    prefix, nodes, qo, Hq, Hkv = s["host"]
    G = Hq // Hkv
    q, o, l = (oracle.as_f64(x) for x in (s["q"], out, lse))
    k, v = (oracle.as_f64(s[x]).reshape(-1, Hkv, q.shape[2]) for x in ("k", "v"))
    for b in range(len(prefix)) if requests is None else requests:
        P, n = prefix[b], nodes[b]
        if n == 0:
            continue
        at = slice(qo[b], qo[b] + n)
        see = np.concatenate([np.ones((n, P), dtype=bool), s["seen"][b]], 1)
        r = s["rows"][b].numpy()
        for h in range(Hkv):
            for g in range(G):
                ref = attend(q[at, h * G + g], k[r, h], v[r, h], s["sm"], see)
                check(o[at, h * G + g], l[at, h * G + g], ref, P + n, BF16, f"request {b} head {h * G + g}")


SHAPES = [
    # prefix, nodes, Hq, Hkv, D, page
    ((1000,), (8,), 32, 8, 128, 16),
    ((0,), (1,), 1, 1, 64, 16),
    ((0, 0, 5), (1, 33, 7), 4, 4, 128, 16),
    ((127, 128, 129, 100, 96), (1, 1, 1, 28, 64), 8, 2, 64, 16),
    ((300, 0, 64, 4000), (16, 5, 1, 12), 32, 8, 128, 16),
    ((500, 10), (64, 40), 32, 8, 128, 16),
    ((200, 700), (65, 130), 8, 4, 64, 32),
    ((50, 260), (300, 150), 16, 1, 128, 64),
    ((100, 3), (33, 34), 14, 2, 64, 8),
    ((77, 140), (20, 31), 6, 3, 128, 24),
    ((333, 1), (17, 2), 16, 8, 128, 1),
    ((60, 700), (129, 9), 5, 5, 64, 3),
    ((1000, 90), (50, 3), 10, 2, 128, 256),
    ((30, 20, 10, 500), (0, 6, 0, 4), 8, 2, 128, 128),
    ((2500,), (1,), 16, 2, 128, 16),
    ((40,), (1024,), 1, 1, 64, 16),
    ((190, 8, 1000), (11, 21, 43), 9, 3, 128, 16),
]


def _ids(s):
    return f"{len(s[0])}x{max(s[0])}+{max(s[1])}-{s[2]}/{s[3]}-D{s[4]}-p{s[5]}"


@pytest.mark.parametrize("kind", ["tree", "random", "chain"])
@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
def test_tree(lib, shape, kind):
    prefix, nodes, Hq, Hkv, D, page = shape
    s = make(sum(prefix) + D, prefix, nodes, Hq, Hkv, D, page, kind)
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_rows_that_see_nothing(lib):
    s = make(1, (0, 0, 0), (40, 3, 130), 8, 2, 64, 16, "none")
    out, lse, err = call(lib, s)
    assert err == 0
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_bits_past_the_request_are_ignored(lib):
    s = make(2, (100, 20), (5, 40), 8, 2, 128, 16, "tree", extra_words=2)
    s["mask"][:5] |= -32  # tokens 5 .. 31 of a request of five
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("scale", [-0.25, 0.0, 3.0])
def test_scales(lib, scale):
    s = make(3, (300, 17), (12, 9), 8, 2, 64, 16)
    s["sm"] = scale
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_many_requests(lib):
    rng = np.random.default_rng(4)
    prefix, nodes = rng.integers(0, 400, 150).tolist(), rng.integers(0, 20, 150).tolist()
    s = make(4, prefix, nodes, 8, 2, 64, 16)
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse, range(0, 150, 7))


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (12, 4, 64)])
def test_many_trees_of_all_sizes(lib, Hq, Hkv, D):
    """More units than CTAs, with one Q tile and with two, in turn on the same CTA; padding rows behind
    the last request are left as they were."""
    rng = np.random.default_rng(14)
    nodes = (2.0 ** rng.uniform(0, 7, 110)).astype(int).tolist()
    prefix = rng.integers(0, 500, 110).tolist()
    s = make(14, prefix, nodes, Hq, Hkv, D, 16)
    N = sum(nodes)
    pad = lambda x, fill: torch.cat([x, torch.full((7,) + x.shape[1:], fill, dtype=x.dtype, device="cuda")])  # noqa: E731
    s["q"], s["mask"] = pad(s["q"], 1.0), pad(s["mask"], -1)
    fill = torch.full_like(s["q"], 7.0)
    out, lse, err = call(lib, s, out=fill)
    assert err == 0
    assert torch.all(out[N:] == 7.0)
    verify(s, out, lse, range(0, 110, 5))
    for _ in range(3):
        o2, l2, _ = call(lib, s)
        assert torch.equal(o2[:N], out[:N]) and torch.equal(l2[:N], lse[:N])


def test_pool_past_32_bits(lib):
    """Pages whose byte offsets pass 4 GB."""
    small = make(15, (300, 40), (20, 9), 8, 8, 128, 16)
    n = small["k"].shape[0]
    first = 150_000  # pages of 32 KB
    k = torch.zeros(first + n, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[first:], v[first:] = small["k"], small["v"]
    out, lse, err = call(lib, small)
    big = dict(small, k=k, v=v, pages=small["pages"] + first)
    o2, l2, err = call(lib, big)
    assert err == 0 and torch.equal(out, o2) and torch.equal(lse, l2)
    # the same cache one row a page (gathers of rows)
    rows = torch.cat([torch.as_tensor(r) for r in small["rows"]]).int().cuda()
    lens = torch.tensor([0, 320, 369], dtype=torch.int32).cuda()
    one = dict(small, k=k.view(-1, 1, 8, 128), v=v.view(-1, 1, 8, 128), pages=rows + first * 16, indptr=lens)
    o3, l3, err = call(lib, one)
    assert err == 0
    verify(small, o3, l3)


def test_growing_scores(lib):
    """Scores that grow along the context: the running maximum moves, O is rescaled in every tile."""
    s = make(5, (3000,), (10,), 8, 2, 128, 16)
    ramp = torch.linspace(0, 12, 3010)
    r = s["rows"][0]
    k = s["k"].view(-1, 2, 128)
    k[r.cuda()] = (ramp[:, None, None] * torch.sign(s["q"][0, :2].float().cpu())[None]).to(torch.bfloat16).cuda()
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_what_a_row_does_not_see_does_not_reach_it(lib):
    """Infinities and NaNs in drafted K and V: rows that do not see them keep their bits."""
    s = make(6, (200, 50), (70, 30), 8, 2, 64, 16, "tree", v_poison=False)
    out, lse, _ = call(lib, s)
    v, k = s["v"].clone(), s["k"].clone()
    inf, nan = float("inf"), float("nan")
    r0, r1 = s["rows"][0], s["rows"][1]
    t0, t1 = 20, 4
    v.view(-1, 2, 64)[r0[200 + t0], 0, 5] = inf
    v.view(-1, 2, 64)[r0[200 + t0], 0, 6] = -inf
    v.view(-1, 2, 64)[r0[200 + t0], 0, 7] = nan
    v.view(-1, 2, 64)[r0[200 + 33], 0, 5] = -inf
    k.view(-1, 2, 64)[r1[50 + t1], 1] = nan
    o2, l2, err = call(lib, dict(s, v=v, k=k))
    assert err == 0
    see0, see33 = (torch.tensor(s["seen"][0][:, t]).cuda() for t in (t0, 33))
    want = out.clone()
    w = want[:70, :4]  # KV head 0
    w[:, :, 5][see0] = inf
    w[:, :, 6][see0] = -inf
    w[:, :, 7][see0] = nan
    w[:, :, 5][see33] = torch.where(see0[see33], nan, -inf).to(w.dtype)[:, None].expand(-1, 4)
    see1 = torch.tensor(s["seen"][1][:, t1]).cuda()
    want[70:, 4:][see1] = nan
    keep = torch.isfinite(want)
    assert torch.equal(torch.isnan(o2), torch.isnan(want))
    assert torch.equal(o2[torch.isinf(want)], want[torch.isinf(want)])
    assert torch.equal(o2[keep], out[keep])  # other dims of the rows that do see them included
    unseen = torch.ones_like(lse, dtype=torch.bool)
    unseen[70:, 4:] &= ~see1[:, None]
    assert torch.equal(l2[unseen], lse[unseen])


def test_errors_are_reported(lib):
    s = make(7, (100, 60), (9, 5), 8, 2, 64, 16)
    ref = call(lib, s)
    assert ref[2] == 0
    pages = s["pages"].clone()
    pages[2] = 10 ** 6
    out, _, err = call(lib, dict(s, pages=pages))
    assert err == lib.DEVERR_PAGE_OOB and torch.equal(out[9:], ref[0][9:])
    out, _, err = call(lib, dict(s, prefix=s["prefix"] + torch.tensor([20, 0], device="cuda", dtype=torch.int32)))
    assert err == lib.DEVERR_LENGTH and torch.equal(out[9:], ref[0][9:])
    out, _, err = call(lib, dict(s, prefix=torch.tensor([-1, 60], device="cuda", dtype=torch.int32)))
    assert err == lib.DEVERR_LENGTH and torch.equal(out[9:], ref[0][9:])
    fill = torch.full_like(s["q"], 7.0)
    out, lse, err = call(lib, dict(s, most=5), out=fill)  # the first request has nine
    assert err == lib.DEVERR_LENGTH and torch.equal(out[9:], ref[0][9:])
    assert torch.all(out[5:9] == 7.0)  # five are covered, and see none of the other four
    prefix, nodes, qo, Hq, Hkv = s["host"]
    five = dict(s, host=((100,), (5,), qo, Hq, Hkv), rows=[s["rows"][0][:105]], seen=[s["seen"][0][:5, :5]])
    verify(five, out, lse)
    out, _, err = call(lib, dict(s, qo=torch.tensor([0, 9, 15], device="cuda", dtype=torch.int32)))
    assert err == lib.DEVERR_ROW_OOB and torch.equal(out[:9], ref[0][:9])


def test_deterministic_and_on_another_stream(lib):
    s = make(8, (5000, 31, 700), (12, 70, 3), 32, 8, 128, 16)
    out, lse, _ = call(lib, s)
    st = torch.cuda.Stream()
    for _ in range(3):
        o2, l2, _ = call(lib, s, stream=st)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_chain_is_the_extend(lib):
    """A chain of drafted tokens is the causal extend: two kernels, within the rounding of both."""
    s = make(9, (130, 900), (60, 17), 32, 8, 128, 16, "chain")
    out, lse, _ = call(lib, s)
    o2, l2 = lib.paged_extend(s["q"], s["k"], s["v"], s["qo"], s["indptr"], s["pages"], s["prefix"], s["most"], s["sm"])
    assert (out.float() - o2.float()).abs().max() <= 2e-2 and (lse - l2).abs().max() <= 1e-4


@pytest.mark.parametrize("nodes", [(1,), (7, 0, 33, 64), (300, 1)])
def test_mask_from_parents(lib, nodes):
    rng = np.random.default_rng(sum(nodes))
    parents, want = [], []
    words = -(-max(nodes) // 32)
    for n in nodes:
        seen = np.zeros((n, n), dtype=bool)
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -3
            parents.append(p)
            seen[i] = seen[p] if p >= 0 else False
            seen[i, i] = True
        want.append(words_of(seen, words) if n else np.zeros((0, words), np.int32))
    qo = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), dtype=torch.int32).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.tree_mask_from_parents(torch.tensor(parents, dtype=torch.int32).cuda(), qo, max(nodes), err_word=err)
    assert int(err) == 0 and np.array_equal(got.cpu().numpy(), np.concatenate(want))


def test_mask_from_parents_reports_bad_parents(lib):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.tree_mask_from_parents(i32([-1, 1, 0, 5]), i32([0, 4]), 4, err_word=err)
    assert int(err) == lib.DEVERR_LENGTH and got.flatten().tolist() == [1, 2, 5, 8]
    err.zero_()
    got = lib.tree_mask_from_parents(i32([-1] * 40), i32([0, 40]), 32, err_word=err)
    assert int(err) == lib.DEVERR_LENGTH and torch.all(got[32:] == 0)
    err.zero_()
    lib.tree_mask_from_parents(i32([-1] * 4), i32([0, 5]), 8, err_word=err)
    assert int(err) == lib.DEVERR_ROW_OOB


def test_mask_from_parents_stops_at_the_longest_tree(lib):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((12, 2), -5, dtype=torch.int32, device="cuda")
    lib.tree_mask_from_parents(i32([-1, 0] + [-1] * 10), i32([0, 2, 12]), 7, out=out, err_word=err)
    assert int(err) == lib.DEVERR_LENGTH
    assert out[:9].tolist() == [[1, 0], [3, 0]] + [[1 << t, 0] for t in range(7)] and torch.all(out[9:] == -5)


@pytest.mark.parametrize("nodes,Hq,Hkv,D", [(30, 8, 2, 128), (50, 8, 2, 128), (60, 8, 2, 64), (5, 8, 2, 128), (12, 8, 2, 64)])
def test_scores_that_jump_within_a_tile(lib, nodes, Hq, Hkv, D):
    """Scores that jump up by a little and by a lot from one run of positions to the next: the reference
    maximum moves between tiles and between the halves of one, weights already written are scaled."""
    n = 1500 + nodes
    s = make(8, (1500,), (nodes,), Hq, Hkv, D, 16)
    rng = np.random.default_rng(nodes)
    level, steps = 0.0, []
    while sum(steps_n for steps_n, _ in steps) < n:
        steps.append((int(rng.integers(5, 90)), level))
        level += float(rng.choice([0.2, 1.0, 4.0, -3.0, 25.0]))
    level = np.concatenate([np.full(c, x) for c, x in steps])[:n]
    k = s["k"].view(-1, Hkv, D)
    turn = torch.sign(s["q"][0, ::Hq // Hkv].float().cpu())[None]
    k[s["rows"][0].cuda()] = (torch.tensor(level, dtype=torch.float32)[:, None, None] * turn / 3).to(torch.bfloat16).cuda()
    out, lse, err = call(lib, s)
    assert err == 0
    verify(s, out, lse)


def test_many_launches_back_to_back(lib):
    """A full queue of launches over ragged trees, eager: every one gives the first one's bits."""
    rng = np.random.default_rng(3)
    prefix, nodes = rng.integers(200, 1500, 48), rng.integers(1, 40, 48)
    s = make(12, [int(p) for p in prefix], [int(n) for n in nodes], 16, 4, 128, 16)
    want, lse, err = call(lib, s)
    assert err == 0
    ws = torch.empty(lib.tree_workspace_size(48, 16, 4, 128, s["most"]), dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, l = torch.empty_like(want), torch.empty_like(lse)
    for _ in range(40):
        for _ in range(50):
            lib.paged_tree_attention(s["q"], s["k"], s["v"], s["qo"], s["indptr"], s["pages"], s["prefix"], s["mask"],
                                     s["most"], s["sm"], out=out, lse=l, workspace=ws, err_word=word)
        wrong += (out != want).sum() + (l != lse).sum()
        out.zero_()
        l.zero_()
    assert int(wrong) == 0 and int(word) == 0
    verify(s, want, lse, requests=[0, 7])


def test_every_launch_of_a_full_queue(lib):
    """2000 launches over ragged trees, 50 in the queue at a time with an output each: all have the first one's
    bits."""
    rng = np.random.default_rng(3)
    prefix, nodes = rng.integers(200, 1500, 48), rng.integers(1, 40, 48)
    s = make(12, [int(p) for p in prefix], [int(n) for n in nodes], 16, 4, 128, 16)
    want, lse, err = call(lib, s)
    assert err == 0
    verify(s, want, lse, requests=[0, 7])
    ws = torch.empty(lib.tree_workspace_size(48, 16, 4, 128, s["most"]), dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    outs, lses = want.new_empty((50,) + want.shape), lse.new_empty((50,) + lse.shape)
    for _ in range(40):
        outs.zero_()
        lses.zero_()
        for i in range(50):
            lib.paged_tree_attention(s["q"], s["k"], s["v"], s["qo"], s["indptr"], s["pages"], s["prefix"], s["mask"],
                                     s["most"], s["sm"], out=outs[i], lse=lses[i], workspace=ws, err_word=word)
        wrong += (outs != want).sum() + (lses != lse).sum()
    assert int(wrong) == 0 and int(word) == 0
