"""The rotary append, the 8-bit cache and the tree attention as a serving step uses them together:
one after the other on the same pool, captured in CUDA graphs, and on two streams at once."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from _attention64 import attend, check
from test_gpu_tree import tree_rows, words_of

pytestmark = pytest.mark.gpu

F16, BF16 = 2.0 ** -11, 2.0 ** -8
HQ, HKV, D, PAGE, PAGES = 16, 4, 128, 16, 96


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32)).cuda()


def tokens(seed, n, hq=HQ):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    return dict(k=rn(n, HKV, D), v=rn(n, HKV, D), q=rn(n, hq, D))


class Cache8:
    """Two requests' pages of an 8-bit cache; every byte of the pool starts as NaN."""

    def __init__(self, lens):
        self.lens = list(lens)
        perm = np.random.default_rng(1).permutation(PAGES)
        self.pages = [perm[: PAGES // 2], perm[PAGES // 2:]]
        shape = (PAGES, PAGE, HKV, D)
        self.pool = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        self.pool += [torch.ones(shape[:3], device="cuda") for _ in range(2)]
        self.indptr, self.indices = i32([0, PAGES // 2, PAGES]), i32(perm)

    def slots(self, b, first, n):
        j = np.arange(first, first + n)
        return self.pages[b][j // PAGE] * PAGE + j % PAGE

    def values(self, at):
        x = cache8.e4m3_values(self.pool[at].view(torch.uint8).cpu().numpy())
        return (x * self.pool[2 + at].double().cpu().numpy()[..., None]).reshape(-1, HKV, D)

    def rows(self, b):
        return self.slots(b, 0, self.lens[b])


def append(lib, c, table, new):
    """Append new[b] tokens' worth of K/V to request b, rotated by their positions; returns rotated Q."""
    t = tokens(sum(c.lens), sum(new))
    slots, pos = [], []
    for b, n in enumerate(new):
        slots.append(c.slots(b, c.lens[b], n))
        pos += range(c.lens[b], c.lens[b] + n)
        c.lens[b] += n
    lib.rotary_kv_append_fp8(*c.pool, t["k"], t["v"], torch.tensor(np.concatenate(slots)).cuda(), i32(pos), table,
                             q=t["q"])
    return t["q"]


def test_decode_steps_over_an_8_bit_cache(lib):
    """Prompt, then decode steps: every step's attention sees what the appends before it wrote."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache8((0, 0))
    append(lib, c, table, (317, 40))
    for step in range(4):
        q = append(lib, c, table, (1, 1))
        out, lse = lib.paged_decode_fp8(q, *c.pool, c.indptr, c.indices, i32(c.lens), D ** -0.5)
        k, v = c.values(0), c.values(1)
        for b in range(2):
            r = c.rows(b)
            for h in range(HKV):
                hs = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                ref = attend(oracle.as_f64(q[b, hs]), k[r, h], v[r, h], D ** -0.5)
                # every row's V scale is the same power of two or a neighbour: the f16 weights' small ones
                # add at most 2^-24 of the largest weight times sum |v8|
                extra = 2.0 ** -24 * ref[4].max(-1)[:, None] * 2 * np.abs(v[r, h]).sum(0)
                check(out[b, hs].double().cpu().numpy(), lse[b, hs].double().cpu().numpy(), ref, c.lens[b], F16,
                      f"step {step} request {b}", extra)


def test_prefill_behind_an_8_bit_prefix(lib):
    """The cached prefix read back as a paged bf16 cache, for the extend that reads one."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache8((0, 0))
    append(lib, c, table, (200, 77))
    q = append(lib, c, table, (50, 19))
    starts = np.concatenate([[0], np.cumsum([-(-n // PAGE) * PAGE for n in c.lens])])
    ko, vo = (torch.full((int(starts[-1]), HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.paged_gather_fp8(*c.pool, c.indptr, c.indices, i32(c.lens), i32(starts), ko, vo)
    pages = i32(np.arange(starts[-1] // PAGE))
    out, lse = lib.paged_extend(q, ko.view(-1, PAGE, HKV, D), vo.view(-1, PAGE, HKV, D), i32([0, 50, 69]),
                                i32(starts // PAGE), pages, i32([200, 77]), 50, D ** -0.5)
    k, v = c.values(0), c.values(1)
    for b, (first, n, prefix) in enumerate(((0, 50, 200), (50, 19, 77))):
        r = c.rows(b)
        seen = np.tril(np.ones((n, prefix + n), dtype=bool), prefix)
        for h in range(HQ):
            ref = attend(oracle.as_f64(q[first: first + n, h]), k[r, h * HKV // HQ], v[r, h * HKV // HQ], D ** -0.5, seen)
            check(out[first: first + n, h].double().cpu().numpy(), lse[first: first + n, h].double().cpu().numpy(), ref,
                  prefix + n, BF16, f"request {b} head {h}")


class TreeStep:
    """A verification step over a bf16 cache: drafted trees rotated and appended, then attended."""

    def __init__(self, seed, prefix=(150, 33), nodes=(13, 40)):
        rng = np.random.default_rng(seed)
        self.prefix, self.nodes = prefix, nodes
        lens = [p + n for p, n in zip(prefix, nodes)]
        need = [-(-n // PAGE) for n in lens]
        gen = torch.Generator().manual_seed(seed)
        self.k = torch.randn(sum(need) + 2, PAGE, HKV, D, generator=gen).to(torch.bfloat16).cuda()
        self.v = torch.randn(sum(need) + 2, PAGE, HKV, D, generator=gen).to(torch.bfloat16).cuda()
        perm = rng.permutation(sum(need) + 2)[: sum(need)]
        starts = np.concatenate([[0], np.cumsum(need)])
        self.indptr, self.indices = i32(starts), i32(perm)
        self.rows = [perm[starts[b] + np.arange(n) // PAGE] * PAGE + np.arange(n) % PAGE for b, n in enumerate(lens)]
        parents, depth, self.seen = [], [], []
        for n in nodes:
            d, p, s = [], [], np.zeros((n, n), dtype=bool)
            for i in range(n):
                p.append(int(rng.integers(max(0, i - 5), i)) if i else -1)
                d.append(d[p[-1]] + 1 if i else 0)
                s[i] = s[p[-1]] if i else False
                s[i, i] = True
            parents += p
            depth.append(d)
            self.seen.append(s)
        self.parents, self.qo = i32(parents), i32(np.concatenate([[0], np.cumsum(nodes)]))
        self.pos = i32(np.concatenate([np.array(d) + p for d, p in zip(depth, prefix)]))
        self.slots = torch.tensor(np.concatenate([r[p:] for r, p in zip(self.rows, prefix)])).cuda()
        self.new = tokens(seed, sum(nodes))
        self.prefix_lens = i32(prefix)
        N = sum(nodes)
        self.mask = torch.zeros(N, 2, dtype=torch.int32, device="cuda")
        self.q_out = torch.empty_like(self.new["q"])
        self.out = torch.empty_like(self.new["q"])
        self.lse = torch.empty(N, HQ, device="cuda")

    def run(self, lib, table, ws, stream=None):
        lib.rotary_kv_append(self.k, self.v, self.new["k"], self.new["v"], self.slots, self.pos, table, q=self.new["q"],
                             q_out=self.q_out, stream=stream)
        lib.tree_mask_from_parents(self.parents, self.qo, max(self.nodes), out=self.mask, stream=stream)
        lib.paged_tree_attention(self.q_out, self.k, self.v, self.qo, self.indptr, self.indices, self.prefix_lens, self.mask,
                                 max(self.nodes), D ** -0.5, out=self.out, lse=self.lse, workspace=ws, stream=stream)

    def verify(self):
        k, v = (oracle.as_f64(x).reshape(-1, HKV, D) for x in (self.k, self.v))
        q, o, l = (oracle.as_f64(x) for x in (self.q_out, self.out, self.lse))
        first = 0
        for b, n in enumerate(self.nodes):
            seen = np.concatenate([np.ones((n, self.prefix[b]), dtype=bool), self.seen[b]], 1)
            for h in range(HQ):
                ref = attend(q[first: first + n, h], k[self.rows[b], h * HKV // HQ], v[self.rows[b], h * HKV // HQ],
                             D ** -0.5, seen)
                check(o[first: first + n, h], l[first: first + n, h], ref, self.prefix[b] + n, BF16, f"request {b} head {h}")
            first += n


def tree_ws(lib):
    return torch.empty(lib.tree_workspace_size(2, HQ, HKV, D, 64), dtype=torch.uint8, device="cuda")


def test_tree_step(lib):
    table = lib.rotary_cos_sin_table(1024, D, 1e6, scaling="yarn", factor=4.0, original_max_position=512)
    s = TreeStep(3)
    s.run(lib, table, tree_ws(lib))
    s.verify()
    # the tokens of the deepest path, as the chain they are, through the decode: the same attention
    b = 1
    leaf = int(np.argmax(s.seen[b].sum(1)))
    path = np.flatnonzero(s.seen[b][leaf])
    at = sum(s.nodes[:b])
    P = s.prefix[b]
    rows = np.concatenate([s.rows[b][:P], s.rows[b][P + path]])
    k, v = (x.view(-1, 1, HKV, D)[torch.tensor(rows).cuda()].contiguous() for x in (s.k, s.v))
    out, lse = lib.paged_decode(s.q_out[at + leaf: at + leaf + 1].contiguous(), k, v, i32([0, len(rows)]),
                                i32(np.arange(len(rows))), i32([len(rows)]), D ** -0.5)
    assert (out.float() - s.out[at + leaf].float()).abs().max() <= 2e-2
    assert (lse - s.lse[at + leaf]).abs().max() <= 1e-4


def test_graphs_that_share_a_workspace(lib):
    """A tree step and an 8-bit decode step, each captured; replayed in turn on the same workspace, with
    new inputs in the captured buffers, they give the eager calls' bits."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    need = max(lib.tree_workspace_size(2, HQ, HKV, D, 64), lib.decode_fp8_workspace_size(2, HQ, HKV, D))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    tree = TreeStep(4)
    c = Cache8((0, 0))
    append(lib, c, table, (300, 55))
    new = tokens(9, 2)
    slots, pos, lens = torch.tensor(np.concatenate([c.slots(0, 300, 1), c.slots(1, 55, 1)])).cuda(), i32([300, 55]), i32([301, 56])
    out, lse = torch.empty(2, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, HQ, device="cuda")
    q_out = torch.empty_like(out)
    starts = i32([0, 304, 360])
    ko, vo = (torch.zeros(360, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = torch.cuda.Stream()

    def decode():
        lib.rotary_kv_append_fp8(*c.pool, new["k"], new["v"], slots, pos, table, q=new["q"], q_out=q_out, stream=st)
        lib.paged_decode_fp8(q_out, *c.pool, c.indptr, c.indices, lens, D ** -0.5, out=out, lse=lse, workspace=ws, stream=st)
        lib.paged_gather_fp8(*c.pool, c.indptr, c.indices, lens, starts, ko, vo, stream=st)

    results = lambda: [x.clone() for x in (tree.out, tree.lse, out, lse, ko, vo)]  # noqa: E731
    st.wait_stream(torch.cuda.current_stream())
    tree.run(lib, table, ws, st)
    decode()
    st.synchronize()
    eager = results()
    graphs = []
    for step in (lambda: tree.run(lib, table, ws, st), decode):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
        graphs.append(g)
    for x in (tree.out, tree.lse, out, lse, ko, vo):
        x.zero_()
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results(), eager))
    # other tokens in the same buffers: the replay follows them
    other = tokens(10, 2)
    for n in new:
        new[n].copy_(other[n])
    tree.new["k"].copy_(tree.new["k"].flip(0))
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    replayed = results()
    tree.run(lib, table, ws, st)
    decode()
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(results(), replayed))
    assert not torch.equal(replayed[2], eager[2]) and not torch.equal(replayed[0], eager[0])
    tree.verify()


def test_two_streams_at_once(lib):
    """Two tree steps on two streams, each with its workspace, many times over."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    steps = [TreeStep(5), TreeStep(6, (700, 20), (9, 64))]
    ws = [tree_ws(lib), tree_ws(lib)]
    for s, w in zip(steps, ws):
        s.run(lib, table, w)
    torch.cuda.synchronize()
    want = [(s.out.clone(), s.lse.clone()) for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for s, w, st in zip(steps, ws, streams):
            s.run(lib, table, w, st)
    torch.cuda.synchronize()
    for s, (o, l) in zip(steps, want):
        assert torch.equal(s.out, o) and torch.equal(s.lse, l)
        s.verify()


def test_binding_refusals_on_the_device(lib):
    """Shapes and types the binding does not pass on."""
    c = Cache8((10, 10))
    q = tokens(1, 2)["q"]
    good = (q, *c.pool, c.indptr, c.indices, i32([10, 10]), 1.0)

    def with_(i, x):
        a = list(good)
        a[i] = x
        return a

    lib.paged_decode_fp8(*good)
    for i, x, error in ((0, q.float(), TypeError), (0, q[:1].contiguous(), ValueError), (0, q[..., :64].contiguous(), ValueError),
                        (0, q.transpose(0, 1), ValueError), (1, c.pool[0].float(), TypeError), (3, c.pool[2].half(), TypeError),
                        (3, c.pool[2][:1].contiguous(), ValueError), (2, c.pool[1][:4].contiguous(), ValueError),
                        (5, i32([0, 48]), ValueError), (6, c.indices.long(), TypeError), (7, torch.tensor([10, 10], dtype=torch.int32), ValueError)):
        with pytest.raises(error):
            lib.paged_decode_fp8(*with_(i, x))
    with pytest.raises(lib.PagedKVError) as e:
        lib.paged_decode_fp8(*good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError):
        lib.paged_decode_fp8(*good, out=torch.empty(3, HQ, D, dtype=torch.bfloat16, device="cuda"))
    s = TreeStep(7)
    args = lambda **k: [k.get(n, v) for n, v in (  # noqa: E731
        ("q", s.q_out), ("k", s.k), ("v", s.v), ("qo", s.qo), ("indptr", s.indptr), ("indices", s.indices),
        ("prefix", s.prefix_lens), ("mask", s.mask), ("most", 64), ("scale", 1.0))]
    lib.paged_tree_attention(*args())
    for bad in (dict(most=65), dict(mask=s.mask[:-1].contiguous()), dict(qo=s.qo[:-1].contiguous()), dict(q=s.q_out[..., :64].contiguous())):
        with pytest.raises(ValueError):
            lib.paged_tree_attention(*args(**bad))
    with pytest.raises(TypeError):
        lib.paged_tree_attention(*args(mask=s.mask.bool()))
    with pytest.raises(lib.PagedKVError) as e:
        lib.paged_tree_attention(*args(most=1025, mask=torch.zeros(53, 40, dtype=torch.int32, device="cuda")))
    assert e.value.status == 2
    torch.cuda.synchronize()


def test_starts_beside_the_kernel_before(lib):
    """The kernels start while the one before them on the stream still runs and wait for it: what long
    kernels, copies and joined streams write just before a call is what it reads, eager and captured."""
    table = lib.rotary_cos_sin_table(1024, D, 1e6)
    c = Cache8((0, 0))
    q = append(lib, c, table, (500, 90))[:2].contiguous()
    n = 1 << 26
    slow, st, st2 = torch.zeros(n, device="cuda"), torch.cuda.Stream(), torch.cuda.Stream()
    lens, qd = i32([0, 0]), torch.zeros_like(q)
    out, lse = torch.empty_like(q), torch.empty(2, HQ, device="cuda")
    ws = torch.empty(lib.decode_fp8_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    want = lib.paged_decode_fp8(q, *c.pool, c.indptr, c.indices, i32(c.lens), 0.1)
    real = i32(c.lens)
    host = torch.tensor(c.lens, dtype=torch.int32).pin_memory()
    tree = TreeStep(11)
    tws = tree_ws(lib)
    tree.run(lib, table, tws)
    torch.cuda.synchronize()
    tree_want = tree.out.clone()
    k0, tq = tree.k.clone(), tree.new["q"].clone()

    def step(how):
        lens.zero_()
        qd.zero_()
        slow.add_(1.0)
        if how == "kernel":
            lens.add_(real)
        elif how == "copy":
            lens.copy_(host, non_blocking=True)
        else:
            st2.wait_stream(st)
            with torch.cuda.stream(st2):
                slow.mul_(0.5)
                lens.copy_(real)
            st.wait_stream(st2)
        qd.copy_(q)
        lib.paged_decode_fp8(qd, *c.pool, c.indptr, c.indices, lens, 0.1, out=out, lse=lse, workspace=ws)
        tree.k.zero_()
        tree.new["q"].zero_()
        slow.add_(1.0)
        tree.k.copy_(k0)
        tree.new["q"].copy_(tq)
        tree.run(lib, table, tws)

    for how in ("kernel", "copy", "join"):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for captured in (False, True):
                out.zero_()
                tree.out.zero_()
                if captured:
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=st):
                        step(how)
                    for _ in range(3):
                        g.replay()
                else:
                    step(how)
                st.synchronize()
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), (how, captured)
                assert torch.equal(tree.out, tree_want), (how, captured)


def test_rewritten_scales_are_seen_at_once(lib):
    """Read-back, append, decode, read-back on one stream, again and again over the same slots: each
    call starts while those before it run, and reads rows and scales that the call before it wrote
    and an earlier one had read."""
    c = Cache8((PAGE * PAGES // 2,) * 2)
    n = sum(c.lens)
    slots = torch.tensor(np.concatenate([c.rows(b) for b in range(2)])).cuda()
    out_indptr, lens = i32([0, n // 2, n]), i32(c.lens)
    data = [tokens(40 + i, n) for i in range(4)]
    for i, t in enumerate(data):
        t["v"] *= 2.0 ** (5 * i)
        t["k"] *= 2.0 ** -i
    q = tokens(7, 2)["q"]
    shape = (n, HKV, D)
    ws = torch.empty(lib.decode_fp8_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    outs = [dict(k0=torch.empty(shape, dtype=torch.bfloat16, device="cuda"), v0=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                 k1=torch.empty(shape, dtype=torch.bfloat16, device="cuda"), v1=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                 o=torch.empty_like(q), lse=torch.empty(2, HQ, device="cuda")) for _ in range(8)]

    def run(wait):
        for i, to in enumerate(outs):
            t = data[i % 4]
            lib.paged_gather_fp8(*c.pool, c.indptr, c.indices, lens, out_indptr, to["k0"], to["v0"])
            wait()
            lib.kv_append_fp8(*c.pool, t["k"], t["v"], slots)
            wait()
            lib.paged_decode_fp8(q, *c.pool, c.indptr, c.indices, lens, 0.1, out=to["o"], lse=to["lse"], workspace=ws)
            wait()
            lib.paged_gather_fp8(*c.pool, c.indptr, c.indices, lens, out_indptr, to["k1"], to["v1"])
            wait()

    lib.kv_append_fp8(*c.pool, data[3]["k"], data[3]["v"], slots)
    run(torch.cuda.synchronize)
    want = [{k: x.clone() for k, x in to.items()} for to in outs]
    for i in range(1, 8):
        assert torch.equal(outs[i]["k0"], outs[i - 1]["k1"]) and torch.equal(outs[i]["v0"], outs[i - 1]["v1"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        for how in ("eager", "captured"):
            for to in outs:
                for x in to.values():
                    x.zero_()
            if how == "eager":
                run(lambda: None)
            else:
                with torch.cuda.graph(g, stream=st):
                    run(lambda: None)
                for _ in range(3):
                    g.replay()
            st.synchronize()
            for to, w in zip(outs, want):
                for k in to:
                    assert torch.equal(to[k], w[k]), (how, k)


def test_calls_checked_in_python_are_the_same(lib, monkeypatch):
    """The binding's native module takes the plain calls; without it the Python checks make the same
    ones, and what the module does not take (here: a whole number for the scale) goes that way."""
    native = lib._load_checked()
    assert native.torch_version == torch.__version__
    table = lib.rotary_cos_sin_table(256, D, 1e6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.decode_fp8_workspace_size(2, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    tws = tree_ws(lib)

    def run(scale):
        c = Cache8((40, 90))
        t = tokens(3, 130)
        slots = torch.tensor(np.concatenate([c.rows(b) for b in range(2)])).cuda()
        lib.kv_append_fp8(*c.pool, t["k"], t["v"], slots, err_word=err)
        q = tokens(4, 2)
        pos, at = i32([40, 90]), torch.tensor([c.slots(0, 40, 1)[0], c.slots(1, 90, 1)[0]]).cuda()
        lens = i32([41, 91])
        q_out = torch.empty_like(q["q"])
        lib.rotary_kv_append_fp8(*c.pool, q["k"], q["v"], at, pos, table, q=q["q"], q_out=q_out, interleaved=True,
                                 err_word=err)
        out, lse = torch.empty_like(q_out), torch.empty(2, HQ, device="cuda")
        got = lib.paged_decode_fp8(q_out, *c.pool, c.indptr, c.indices, lens, scale, out=out, lse=lse, workspace=ws,
                                   err_word=err)
        assert got[0] is out and got[1] is lse
        k, v = (torch.zeros(132, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.paged_gather_fp8(*c.pool, c.indptr, c.indices, lens, i32([0, 41, 132]), k, v, err_word=err)
        step = TreeStep(5)
        step.run(lib, table, tws)
        kb, vb = (torch.zeros(PAGES, PAGE, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.rotary_kv_append(kb, vb, q["k"], q["v"], at, pos, table, q=q["q"], err_word=err)
        return [x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x
                for x in (*c.pool, q_out, out, lse, k, v, step.out, kb, vb, q["q"])]

    calls = []

    class Counting:
        def __getattr__(self, name):
            def call(*args):
                status = getattr(native, name)(*args)
                calls.append((name, status))
                return status
            return call

    monkeypatch.setattr(lib, "_checked", Counting())
    want = run(0.125)
    assert {name for name, _ in calls} == {"kv_append_fp8", "rotary_kv_append_fp8", "paged_decode_fp8", "paged_gather_fp8",
                                           "rotary_kv_append", "paged_tree_attention"}
    assert all(status == 0 for _, status in calls)
    calls.clear()
    one = run(1)
    assert ("paged_decode_fp8", None) in calls
    monkeypatch.setattr(lib, "_checked", lib._CheckedInPython())
    for a, b in ((want, run(0.125)), (one, run(1))):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert int(err) == 0
