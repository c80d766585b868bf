"""The 4-bit cache and the movements of rows as a serving step uses them together, and beside the tree attention: one
after the other on the same pool, captured in CUDA graphs, and on two streams at once."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache4
from _attention64 import attend, check
from test_gpu_operators_together import BF16, D, F16, HKV, HQ, PAGE, PAGES, TreeStep, i32, tokens, tree_ws

pytestmark = pytest.mark.gpu

KG, VG = 0.004, 0.002
SCALES = dict(k_global=KG, v_global=VG)


class Cache4:
    """Two requests' pages of a 4-bit cache, and some spare ones; every scale of the pool starts as NaN."""

    def __init__(self, lens, seed=1):
        self.lens = list(lens)
        perm = np.random.default_rng(seed).permutation(PAGES)
        half = PAGES // 2 - 4
        self.pages = [perm[:half].copy(), perm[half: 2 * half].copy()]
        self.spare = perm[2 * half:]
        head = (PAGES, PAGE, HKV)
        self.pool = [torch.zeros(*head, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.pool += [torch.full((*head, D // 16), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                      for _ in range(2)]

    @property
    def indptr(self):
        return i32([0, len(self.pages[0]), len(self.pages[0]) + len(self.pages[1])])

    @property
    def indices(self):
        return i32(np.concatenate(self.pages))

    def slots(self, b, first, n):
        j = np.arange(first, first + n)
        return self.pages[b][j // PAGE] * PAGE + j % PAGE

    def values(self, at):
        x = cache4.values(self.pool[at].cpu().numpy(), self.pool[2 + at].view(torch.uint8).cpu().numpy(), (KG, VG)[at])
        return x.reshape(-1, HKV, D)

    def rows(self, b):
        return self.slots(b, 0, self.lens[b])


def append(lib, c, table, new):
    """Append new[b] tokens' worth of K/V to request b, rotated by their positions; returns rotated Q."""
    t = tokens(sum(c.lens) + 7, sum(new))
    slots, pos = [], []
    for b, n in enumerate(new):
        slots.append(c.slots(b, c.lens[b], n))
        pos += range(c.lens[b], c.lens[b] + n)
        c.lens[b] += n
    lib.rotary_kv_append_fp4(*c.pool, t["k"], t["v"], torch.tensor(np.concatenate(slots)).cuda(), i32(pos), table,
                             q=t["q"], **SCALES)
    return t["q"]


def verify_decode(c, q, out, lse, what):
    k, v = c.values(0), c.values(1)
    for b in range(2):
        r = c.rows(b)
        for h in range(HKV):
            hs = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
            ref = attend(oracle.as_f64(q[b, hs]), k[r, h], v[r, h], D ** -0.5)
            extra = 2.0 ** -32 * ref[4].max(-1)[:, None] * np.abs(v[r, h]).sum(0)  # weights that are subnormal in f16
            check(out[b, hs].double().cpu().numpy(), lse[b, hs].double().cpu().numpy(), ref, c.lens[b], F16,
                  f"{what} request {b}", extra)


def test_decode_steps_and_a_fork(lib):
    """Prompt, decode steps; then the second request becomes a fork of the first, whose begun page is copied, and both
    go on: every step's attention sees what the calls before it wrote."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache4((0, 0))
    append(lib, c, table, (315, 40))
    for step in range(3):
        q = append(lib, c, table, (1, 1))
        out, lse = lib.paged_decode_fp4(q, *c.pool, c.indptr, c.indices, i32(c.lens), D ** -0.5, **SCALES)
        verify_decode(c, q, out, lse, f"step {step}")
    whole, begun = divmod(c.lens[0], PAGE)
    assert 0 < begun < PAGE
    own = c.spare[0]
    lib.copy_pages(c.pool, i32([c.pages[0][whole]]), i32([own]), rows=i32([begun]))
    c.pages[1][:whole] = c.pages[0][:whole]
    c.pages[1][whole] = own
    c.lens[1] = c.lens[0]
    for step in range(3):
        q = append(lib, c, table, (1, 1))
        out, lse = lib.paged_decode_fp4(q, *c.pool, c.indptr, c.indices, i32(c.lens), D ** -0.5, **SCALES)
        verify_decode(c, q, out, lse, f"behind the fork {step}")
    assert not torch.equal(out[0], out[1])


def test_prefill_behind_a_4_bit_prefix(lib):
    """The cached prefix read back as a paged bf16 cache, for the extend that reads one."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache4((0, 0))
    append(lib, c, table, (200, 77))
    q = append(lib, c, table, (50, 19))
    starts = np.concatenate([[0], np.cumsum([-(-n // PAGE) * PAGE for n in c.lens])])
    ko, vo = (torch.full((int(starts[-1]), HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.paged_gather_fp4(*c.pool, c.indptr, c.indices, i32(c.lens), i32(starts), ko, vo, **SCALES)
    out, lse = lib.paged_extend(q, ko.view(-1, PAGE, HKV, D), vo.view(-1, PAGE, HKV, D), i32([0, 50, 69]),
                                i32(starts // PAGE), i32(np.arange(starts[-1] // PAGE)), i32([200, 77]), 50, D ** -0.5)
    # the extend reads the values' bf16
    k, v = (torch.tensor(c.values(at)).float().to(torch.bfloat16).double().numpy() for at in range(2))
    for b, (first, n, prefix) in enumerate(((0, 50, 200), (50, 19, 77))):
        r = c.rows(b)
        seen = np.tril(np.ones((n, prefix + n), dtype=bool), prefix)
        for h in range(HQ):
            ref = attend(oracle.as_f64(q[first: first + n, h]), k[r, h * HKV // HQ], v[r, h * HKV // HQ], D ** -0.5, seen)
            check(out[first: first + n, h].double().cpu().numpy(), lse[first: first + n, h].double().cpu().numpy(), ref,
                  prefix + n, BF16, f"request {b} head {h}")


def test_accepted_path_of_a_tree(lib):
    """Verify a tree, accept the deepest path, move it behind the prefix: the decode over the request is the attention of
    that path's last token."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    s = TreeStep(3)
    s.run(lib, table, tree_ws(lib))
    leaves = [int(np.argmax(seen.sum(1))) for seen in s.seen]
    paths = [np.flatnonzero(seen[leaf]) for seen, leaf in zip(s.seen, leaves)]
    assert all(len(p) > 2 and np.any(p != np.arange(len(p))) for p in paths)
    starts = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
    # the lists hold each request's drafted positions too
    lib.compact_accepted([s.k, s.v], s.indptr, s.indices, s.prefix_lens, i32(starts), i32(np.concatenate(paths)))
    at = np.array([0, s.nodes[0]]) + leaves
    q = s.q_out[torch.tensor(at).cuda()].contiguous()
    lens = [p + len(path) for p, path in zip(s.prefix, paths)]
    out, lse = lib.paged_decode(q, s.k, s.v, s.indptr, s.indices, i32(lens), D ** -0.5)
    want, want_lse = s.out[torch.tensor(at).cuda()], s.lse[torch.tensor(at).cuda()]
    # both are within a bf16 rounding of the weights and of the result of the same attention
    assert (out.float() - want.float()).abs().max() <= 2e-2
    assert (lse - want_lse).abs().max() <= 1e-4


def test_graphs_that_share_a_workspace(lib):
    """A 4-bit decode step with copies and a read-back, and an 8-bit one's workspace: captured, replayed with new inputs in
    the captured buffers, it gives the eager calls' bits."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    need = lib.decode_fp4_workspace_size(2, HQ, HKV, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    c = Cache4((0, 0))
    append(lib, c, table, (300, 55))
    new = tokens(9, 2)
    slots, pos, lens = torch.tensor(np.concatenate([c.slots(0, 300, 1), c.slots(1, 55, 1)])).cuda(), i32([300, 55]), i32([301, 56])
    out, lse = torch.empty(2, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, HQ, device="cuda")
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    q_out = torch.empty_like(out)
    starts = i32([0, 304, 360])
    ko, vo = (torch.zeros(360, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    indptr, indices = c.indptr, c.indices
    src, dst, rows = i32([c.pages[0][18], c.pages[1][3]]), i32(c.spare[:2]), i32([13, 8])
    swapped = np.concatenate(c.pages).copy()
    swapped[18], swapped[len(c.pages[0]) + 3] = c.spare[:2]
    swapped = i32(swapped)
    moved_starts, moved = i32([0, 2, 3]), i32([1, 3, 2])
    prefix = i32([296, 52])
    st = torch.cuda.Stream()

    def step():
        lib.rotary_kv_append_fp4(*c.pool, new["k"], new["v"], slots, pos, table, q=new["q"], q_out=q_out, **SCALES, stream=st)
        lib.paged_decode_fp4(q_out, *c.pool, indptr, indices, lens, D ** -0.5, out=out, lse=lse, workspace=ws, **SCALES,
                             stream=st)
        lib.copy_pages(c.pool, src, dst, rows=rows, stream=st)
        lib.compact_accepted(c.pool, indptr, swapped, prefix, moved_starts, moved, stream=st)
        lib.paged_decode_fp4(q_out, *c.pool, indptr, swapped, lens, D ** -0.5, out=out2, lse=lse2, workspace=ws, **SCALES,
                             stream=st)
        lib.paged_gather_fp4(*c.pool, indptr, swapped, lens, starts, ko, vo, **SCALES, stream=st)

    results = lambda: [x.clone() for x in (out, lse, out2, lse2, ko, vo)]  # noqa: E731
    st.wait_stream(torch.cuda.current_stream())
    step()
    st.synchronize()
    eager = results()
    assert not torch.equal(out, out2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    for x in (out, lse, out2, lse2, ko, vo):
        x.zero_()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results(), eager))
    other = tokens(10, 2)
    for n in new:
        new[n].copy_(other[n])
    g.replay()
    torch.cuda.synchronize()
    replayed = results()
    step()
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(results(), replayed))
    assert not torch.equal(replayed[0], eager[0])


def test_two_streams_at_once(lib):
    """Decodes on two streams, each with its workspace, many times over."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    steps = []
    for seed, new in ((1, (600, 9)), (2, (33, 500))):
        c = Cache4((0, 0), seed)
        q = append(lib, c, table, new)[:2].contiguous()
        steps.append(dict(c=c, q=q, lens=i32(c.lens), indptr=c.indptr, indices=c.indices, out=torch.empty_like(q),
                          lse=torch.empty(2, HQ, device="cuda"), st=torch.cuda.Stream(),
                          ws=torch.empty(lib.decode_fp4_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")))

    def run(s, st):
        lib.paged_decode_fp4(s["q"], *s["c"].pool, s["indptr"], s["indices"], s["lens"], D ** -0.5, out=s["out"],
                             lse=s["lse"], workspace=s["ws"], **SCALES, stream=st)

    for s in steps:
        run(s, None)
    torch.cuda.synchronize()
    want = [(s["out"].clone(), s["lse"].clone()) for s in steps]
    for _ in range(20):
        for s in steps:
            run(s, s["st"])
    torch.cuda.synchronize()
    for s, (o, l) in zip(steps, want):
        assert torch.equal(s["out"], o) and torch.equal(s["lse"], l)
        verify_decode(s["c"], s["q"], s["out"], s["lse"], "streams")


def test_starts_beside_the_kernel_before(lib):
    """What long kernels and copies write just before a call is what it reads, eager and captured: lengths, queries, page lists
    and rows, for every call of this part."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache4((0, 0))
    q = append(lib, c, table, (500, 90))[:2].contiguous()
    n = 1 << 26
    slow, st = torch.zeros(n, device="cuda"), torch.cuda.Stream()
    t = tokens(5, 2)
    slots, pos = torch.tensor([c.spare[0] * PAGE, c.spare[0] * PAGE + 5]).cuda(), i32([7, 9])
    live = dict(lens=i32(c.lens), q=q, indices=c.indices, src=i32([c.pages[0][3]]), dst=i32([c.spare[1]]), prefix=i32([490, 80]),
                taken=i32([2, 5, 1]), k=t["k"], slots=slots)
    now = {k: torch.zeros_like(v) for k, v in live.items()}
    indptr, starts, moved = c.indptr, i32([0, 504, 600]), i32([0, 2, 3])
    out, lse = torch.empty_like(q), torch.empty(2, HQ, device="cuda")
    ko, vo = (torch.zeros(600, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(lib.decode_fp4_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    before = [x.clone() for x in c.pool]

    def step(slowly):
        for x, b in zip(c.pool, before):
            x.copy_(b)
        for call in ("append", "copy", "compact", "decode", "gather"):
            if slowly:
                for k, v in now.items():
                    v.zero_()
                slow.add_(1.0)
            for k, v in now.items():
                v.copy_(live[k])
            if call == "append":
                lib.kv_append_fp4(*c.pool, now["k"], t["v"], now["slots"], **SCALES)
            elif call == "copy":
                lib.copy_pages(c.pool, now["src"], now["dst"])
            elif call == "compact":
                lib.compact_accepted(c.pool, indptr, now["indices"], now["prefix"], moved, now["taken"])
            elif call == "decode":
                lib.paged_decode_fp4(now["q"], *c.pool, indptr, now["indices"], now["lens"], 0.1, out=out, lse=lse,
                                     workspace=ws, **SCALES)
            else:
                lib.paged_gather_fp4(*c.pool, indptr, now["indices"], now["lens"], starts, ko, vo, **SCALES)

    def results():
        return [x.clone() for x in (out, lse, ko, vo, c.pool[0], c.pool[1], c.pool[2].view(torch.uint8), c.pool[3].view(torch.uint8))]

    torch.cuda.synchronize()
    step(False)
    torch.cuda.synchronize()
    want = results()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(True)
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step(True)
        for _ in range(3):
            out.zero_(), ko.zero_()
            g.replay()
            st.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(results(), want))


BUSY = 40_000_000  # cycles, about 20 ms


def test_a_workspace_is_not_handed_on_before_the_call_is_done(lib):
    """Calls in a row on a side stream without a wait, while the current stream allocates and overwrites blocks of the
    sizes that the calls use."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache4((0, 0))
    q = append(lib, c, table, (600, 90))[:2].contiguous()
    args = (q, *c.pool, c.indptr, c.indices, i32(c.lens), 0.1)
    size = lib.decode_fp4_workspace_size(2, HQ, HKV, D)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = lib.paged_decode_fp4(*args, **SCALES)
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(st):
            torch.cuda._sleep(BUSY // 200)
        got.append(lib.paged_decode_fp4(*args, **SCALES, stream=st))
        for _ in range(3):
            torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")
            torch.full_like(want[0], float("nan"))
            torch.full_like(want[1], float("nan"))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_binding_refusals_on_the_device(lib):
    """Shapes and types the binding does not pass on."""
    c = Cache4((10, 10))
    q = tokens(1, 2)["q"]
    good = (q, *c.pool, c.indptr, c.indices, i32([10, 10]), 1.0)

    def with_(i, x):
        a = list(good)
        a[i] = x
        return a

    lib.paged_decode_fp4(*good)
    for i, x, error in ((0, q.float(), TypeError), (0, q[:1].contiguous(), ValueError), (0, q[..., :64].contiguous(), ValueError),
                        (0, q.transpose(0, 1), ValueError), (1, c.pool[0].float(), TypeError), (3, c.pool[2].float(), TypeError),
                        (3, c.pool[2][:1].contiguous(), ValueError), (2, c.pool[1][:4].contiguous(), ValueError),
                        (3, c.pool[2][..., :4].contiguous(), ValueError), (4, c.pool[3].view(torch.uint8), TypeError),
                        (5, i32([0, 44]), ValueError), (6, c.indices.long(), TypeError),
                        (7, torch.tensor([10, 10], dtype=torch.int32), ValueError)):
        with pytest.raises(error):
            lib.paged_decode_fp4(*with_(i, x))
    for bad in (dict(k_global=0.0), dict(v_global=-1.0), dict(k_global=float("nan")), dict(v_global=1e30)):
        with pytest.raises(lib.PagedKVError, match="invalid"):
            lib.paged_decode_fp4(*good, **bad)
    with pytest.raises(lib.PagedKVError) as e:
        lib.paged_decode_fp4(*good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError):
        lib.paged_decode_fp4(*good, out=torch.empty(3, HQ, D, dtype=torch.bfloat16, device="cuda"))
    t, slots = tokens(2, 4), torch.arange(4).cuda()
    with pytest.raises(ValueError, match="num_tokens"):
        lib.kv_append_fp4(*c.pool, t["k"], t["v"], slots[:3].contiguous())
    with pytest.raises(ValueError, match="rotary_dim"):
        lib.rotary_kv_append_fp4(*c.pool, t["k"], t["v"], slots, slots.int(), torch.zeros(8, 130, device="cuda"))
    with pytest.raises(ValueError, match="num_out_rows"):
        lib.paged_gather_fp4(*c.pool, c.indptr, c.indices, i32([4, 4]), i32([0, 4, 8]), t["k"][:, :2].contiguous(), t["v"])
    torch.cuda.synchronize()


def test_calls_checked_in_python_are_the_same(lib, monkeypatch):
    """The binding's native module takes the plain calls; without it the Python checks make the same ones, and what the
    module does not take (here: whole numbers for scales) goes that way."""
    native = lib._load_checked()
    table = lib.rotary_cos_sin_table(256, D, 1e6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.decode_fp4_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")

    def run(g):
        c = Cache4((40, 90))
        for x in c.pool[2:]:
            x.zero_()
        t = tokens(3, 130)
        slots = torch.tensor(np.concatenate([c.rows(b) for b in range(2)])).cuda()
        lib.kv_append_fp4(*c.pool, t["k"], t["v"], slots, err_word=err, k_global=g, v_global=g)
        q = tokens(4, 2)
        pos, at = i32([40, 90]), torch.tensor([c.slots(0, 40, 1)[0], c.slots(1, 90, 1)[0]]).cuda()
        lens = i32([41, 91])
        q_out = torch.empty_like(q["q"])
        lib.rotary_kv_append_fp4(*c.pool, q["k"], q["v"], at, pos, table, q=q["q"], q_out=q_out, interleaved=True,
                                 err_word=err, k_global=g, v_global=g)
        lib.copy_pages(tuple(c.pool), i32([c.pages[0][2]]), i32([c.spare[0]]), rows=i32([9]), err_word=err)
        lib.compact_accepted(c.pool, c.indptr, c.indices, i32([30, 80]), i32([0, 2, 3]), i32([1, 4, 2]), err_word=err)
        out, lse = torch.empty_like(q_out), torch.empty(2, HQ, device="cuda")
        got = lib.paged_decode_fp4(q_out, *c.pool, c.indptr, c.indices, lens, 0.125, out=out, lse=lse, workspace=ws,
                                   err_word=err, k_global=g, v_global=g)
        assert got[0] is out and got[1] is lse
        k, v = (torch.zeros(132, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.paged_gather_fp4(*c.pool, c.indptr, c.indices, lens, i32([0, 41, 132]), k, v, err_word=err, k_global=g, v_global=g)
        return [x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x for x in (*c.pool, q_out, out, lse, k, v)]

    calls = []

    class Counting:
        def __getattr__(self, name):
            def call(*args):
                status = getattr(native, name)(*args)
                calls.append((name, status))
                return status
            return call

    monkeypatch.setattr(lib, "_checked", Counting())
    want = run(0.25)
    assert [name for name, _ in calls] == ["kv_append_fp4", "rotary_kv_append_fp4", "copy_pages", "compact_accepted",
                                           "paged_decode_fp4", "paged_gather_fp4"]
    assert all(status == 0 for _, status in calls)
    calls.clear()
    one = run(1)
    assert ("paged_decode_fp4", None) in calls and ("copy_pages", 0) in calls
    monkeypatch.setattr(lib, "_checked", lib._CheckedInPython())
    for a, b in ((want, run(0.25)), (one, run(1))):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert int(err) == 0
