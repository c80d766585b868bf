"""Compaction where a warp takes runs of two to four chunks, and the accepted path of a verified tree row by row.  Bytes move, so
nothing here has a tolerance but the attention, whose bound is _attention64's."""

import numpy as np
import pytest
import torch

import oracle
from _attention64 import attend, check
from test_gpu_operators_together import BF16, D, HKV, HQ, TreeStep, i32, tree_ws
from test_gpu_page_ops import trees

pytestmark = pytest.mark.gpu

CHUNK = 32  # pieces that a warp takes side by side
WARPS = 32  # that an SM has room for

# the bytes of a slot of each tensor, and what the first bytes of the tensors lie behind a multiple of 16
SETS = {
    "bf16 8x128, 36 layers": ([2048] * 72, 0),
    "of all widths": ([2048, 1024, 512, 64, 32, 16, 1040, 528, 496, 2032, 4112] * 3, 0),
    "ending in a narrow one": ([512, 1024, 16], 0),
    "narrow": ([256, 64, 16, 496, 128] * 4 + [16], 0),
    "4 bits 1x64": ([32, 32, 4, 4] * 9, 0),
    "of all pieces": ([1024, 24, 4, 2, 1, 33, 520, 2048, 1028, 130] * 2, 0),
    "off by 8": ([1024, 64, 256, 2048, 520], 8),
    "off by 1": ([96, 16, 33], 1),
}


def chunks_of(slots, shift):
    piece = lambda n: next(p for p in (16, 8, 4, 2, 1) if n % p == 0 and shift % p == 0)  # noqa: E731
    return sum(-(-(n // piece(n)) // CHUNK) for n in slots)


def tensors_of(slots, shift, num_pages, page):
    out = []
    for i, n in enumerate(slots):
        gen = torch.Generator(device="cuda").manual_seed(i)
        size = num_pages * page * n
        raw = torch.randint(0, 256, (size + 16,), generator=gen, device="cuda", dtype=torch.uint8)
        out.append(raw[shift: shift + size].view(num_pages, page, n))
    return out


def compact_and_check(lib, tensors, t, page):
    src, dst = (torch.tensor(t[x]).cuda() for x in ("src", "dst"))
    want = []
    for x in tensors:
        w = x.clone().view(-1, x.shape[2])
        w[dst] = w[src]  # the right side is read first
        want.append(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.compact_accepted(tensors, *t["args"], err_word=err)
    assert int(err) == 0
    for i, (x, w) in enumerate(zip(tensors, want)):
        assert torch.equal(x.view(w.shape), w), f"tensor {i} of {x.shape[2]} bytes a slot"


@pytest.mark.parametrize("run", [1, 2, 3, 4, 9])
@pytest.mark.parametrize("kind", SETS)
def test_runs_of_chunks(lib, kind, run):
    """As many trees as give a warp `run` chunks (at most four)."""
    slots, shift = SETS[kind]
    places = torch.cuda.get_device_properties(0).multi_processor_count * WARPS
    chunks = chunks_of(slots, shift)
    B = max(1, ((run - 1) * places + places // 3) // chunks)
    assert run > 4 or -(-B * chunks // places) == run
    page = 4 if B > 100 else 16
    t = trees(np.random.default_rng(run), B, 9, page, 6)
    compact_and_check(lib, tensors_of(slots, shift, t["num_pages"], page), t, page)


@pytest.mark.parametrize("nodes,B", [(80, 70), (300, 20)])
@pytest.mark.parametrize("kind", ["bf16 8x128, 36 layers", "of all widths", "narrow", "of all pieces"])
def test_many_rows_of_a_tree(lib, kind, nodes, B):
    """More accepted rows than a warp has lanes, most of them moving by a few positions."""
    slots, shift = SETS[kind]
    if len(slots) > 40:
        slots, B = slots[:30], B // 2
    rng = np.random.default_rng(nodes)
    t = trees(rng, B, nodes, 16, 20)
    t2 = trees(rng, B, nodes, 16, 20)
    tensors = tensors_of(slots, shift, max(t["num_pages"], t2["num_pages"]), 16)
    compact_and_check(lib, tensors, t, 16)
    compact_and_check(lib, tensors, t2, 16)


def test_64_trees_in_36_layers(lib):
    """Drafted trees of 16 in every layer's bf16 K and V: four chunks a warp."""
    t = trees(np.random.default_rng(64), 64, 16, 16, 40)
    compact_and_check(lib, tensors_of([2048] * 72, 0, t["num_pages"], 16), t, 16)


@pytest.mark.parametrize("seed", [3, 5])
def test_accepted_path_row_by_row(lib, seed):
    """Verify a tree, accept its deepest path, move it behind the prefix: every row of K and of V is where it belongs, the others of
    the prefix are what they were, and the decode is the attention of those rows."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    s = TreeStep(seed)
    s.run(lib, table, tree_ws(lib))
    leaves = [int(np.argmax(seen.sum(1))) for seen in s.seen]
    paths = [np.flatnonzero(seen[leaf]) for seen, leaf in zip(s.seen, leaves)]
    assert all(len(p) > 2 and np.any(p != np.arange(len(p))) for p in paths)
    starts = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
    before = [x.clone().view(-1, HKV, D) for x in (s.k, s.v)]
    lib.compact_accepted([s.k, s.v], s.indptr, s.indices, s.prefix_lens, i32(starts), i32(np.concatenate(paths)))
    lens = [p + len(path) for p, path in zip(s.prefix, paths)]
    k, v = (x.view(-1, HKV, D) for x in (s.k, s.v))
    took = [np.concatenate([r[:p], r[p + path]]) for r, p, path in zip(s.rows, s.prefix, paths)]
    for b, n in enumerate(lens):
        for now, was in zip((k, v), before):
            assert torch.equal(now[torch.tensor(s.rows[b][:n]).cuda()], was[torch.tensor(took[b]).cuda()])
    q = s.q_out[torch.tensor(np.array([0, s.nodes[0]]) + leaves).cuda()].contiguous()
    out, lse = lib.paged_decode(q, s.k, s.v, s.indptr, s.indices, i32(lens), D ** -0.5)
    kd, vd = (oracle.as_f64(x) for x in before)
    for b, n in enumerate(lens):
        for h in range(HQ):
            ref = attend(oracle.as_f64(q)[b, h: h + 1], kd[took[b], h * HKV // HQ], vd[took[b], h * HKV // HQ], D ** -0.5)
            check(oracle.as_f64(out)[b, h: h + 1], oracle.as_f64(lse)[b, h: h + 1], ref, n, BF16, f"request {b} head {h}")
