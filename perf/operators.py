"""Cases for the rotary append, the 8-bit KV cache and the attention over drafted trees.

Five operators over a paged KV pool, in their plain form (elementary torch operations in 32 bits) and
as calls of the library:

  rotary        rotate K and Q by their positions, half or interleaved pairs, all or part of the head,
                and write K/V into the pool through a slot mapping
  append8       quantise K/V rows to e4m3 with one power-of-two scale per row and head as they are
                written (with the rotation in front where the case has a rotary width)
  gather8       read an 8-bit cache back as bf16 rows in position order
  decode8       one query per request over an 8-bit paged cache
  tree          every node of a tree of drafted tokens over the cached prefix and its own ancestors

``prepare`` makes the pool, page lists and new rows of one layer's step from the seed; ``run`` is one
call; ``exact`` states the same in 64 bits.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step of a small model: four new tokens, latency alone counts
        dict(name="rotary step of 4, D 64", op="rotary", tokens=4, pad=0, q_heads=14, kv_heads=2,
             head_dim=64, page=16, rotary=64, interleaved=False),
        # a long prompt's prefill in one call, an odd count, neighbouring pairs over half of the head
        dict(name="rotary prefill 8191, partial", op="rotary", tokens=8191, pad=5, q_heads=32, kv_heads=8,
             head_dim=128, page=16, rotary=64, interleaved=True),
        # the append of a decode batch into a page-size-1 cache, without a rotation
        dict(name="append8 step of 32", op="append8", tokens=32, pad=0, q_heads=0, kv_heads=8,
             head_dim=128, page=1, rotary=0, interleaved=False),
        # the append of a mixed step: 256 decodes and four 512-token prefill chunks, rotation fused
        dict(name="append8 mixed step 2304, rotary", op="append8", tokens=2304, pad=0, q_heads=32,
             kv_heads=8, head_dim=128, page=16, rotary=128, interleaved=False),
        # cached prefixes of sixteen requests read back as bf16 for a prefill behind them
        dict(name="gather8 16 prefixes", op="gather8", batch=16, len_min=1, len_max=4096, q_heads=0,
             kv_heads=8, head_dim=128, page=16),
        # four short requests of a small model
        dict(name="decode8 4 short, D 64", op="decode8", batch=4, len_min=38, len_max=512, q_heads=14,
             kv_heads=2, head_dim=64, page=16),
        # a decode batch over a page-size-1 cache
        dict(name="decode8 32, page 1", op="decode8", batch=32, len_min=100, len_max=640, q_heads=16,
             kv_heads=8, head_dim=128, page=1),
        # eight long contexts: every request is split over many SMs
        dict(name="decode8 8 x 32K", op="decode8", batch=8, len_min=32768, len_max=32768, q_heads=32,
             kv_heads=8, head_dim=128, page=16),
        # the decodes of a large continuous batch
        dict(name="decode8 256, ragged", op="decode8", batch=256, len_min=512, len_max=4096, q_heads=32,
             kv_heads=8, head_dim=128, page=16),
        # one user's tree of eight drafted tokens: latency
        dict(name="tree 1 x 8", op="tree", batch=1, nodes_min=8, nodes_max=8, len_min=1000, len_max=1000,
             q_heads=32, kv_heads=8, head_dim=128, page=16),
        # a speculative step of 64 requests, trees of up to sixteen nodes
        dict(name="tree 64 x 16, ragged", op="tree", batch=64, nodes_min=1, nodes_max=16, len_min=512,
             len_max=4096, q_heads=32, kv_heads=8, head_dim=128, page=16),
        # wide trees over long contexts
        dict(name="tree 4 x 64 over 32K", op="tree", batch=4, nodes_min=64, nodes_max=64, len_min=32700,
             len_max=32700, q_heads=32, kv_heads=8, head_dim=128, page=16),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append8", "gather8", "decode8", "decode8", "tree", "tree"])
    kv_heads, group = rng.choice([(1, 8), (2, 7), (2, 16), (3, 2), (4, 5), (4, 8), (8, 1), (8, 2), (8, 4), (16, 1)])
    head_dim = rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 16, 16, 32, 64, 24])
    base = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
    row = kv_heads * head_dim  # values of one token's K
    if op in ("rotary", "append8"):
        tokens = _log_between(rng, 1, 8191)
        base["tokens"] = tokens
        base["pad"] = rng.choice([0, 0, tokens // 7])
        base["rotary"] = rng.choice([16, 32, 48, 64, head_dim])
        base["interleaved"] = rng.random() < 0.5
        if op == "append8" and rng.random() < 0.5:
            base.update(rotary=0, interleaved=False, q_heads=0)
        return base
    most = 400_000 * 1024 // row  # cached tokens of one case
    longest = _log_between(rng, 1, 65536)
    base["len_max"] = longest
    base["len_min"] = max(1, longest - rng.randrange(longest))
    if op == "tree":
        base["nodes_max"] = _log_between(rng, 1, 128)
        base["nodes_min"] = rng.randint(1, base["nodes_max"])
        # scores of one pass stay within the largest listed case's
        most = min(most, 4 * 64 * 32 * 32768 // (base["nodes_max"] * base["q_heads"]))
    base["batch"] = _log_between(rng, 1, max(1, min(512, most // longest)))
    return base


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers evenly over [lo, hi]: their sum does not depend on the seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case, seed):
    lens = _spread(case["len_min"], case["len_max"], case["batch"])
    random.Random(seed).shuffle(lens)
    return lens


def _nodes(case):
    return _spread(case["nodes_min"], case["nodes_max"], case["batch"])


def _power_of_two(k):
    """2^k in fp32 for whole k in [-126, 127], from its bits."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantised(x):
    """e4m3 values and the power-of-two scale of every row (the last axis) of x, in fp32."""
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    mant, exp = torch.frexp(amax)  # amax = mant * 2^exp, mant in [0.5, 1)
    k = torch.where(mant <= 0.875, exp - 9, exp - 8)  # the smallest k with amax <= 448 * 2^k
    k = torch.where(amax > 0, k, -126).clamp(min=-126)
    return (x * _power_of_two(-k).unsqueeze(-1)).to(E4M3), _power_of_two(k)


def _channels(gen, case, dev):
    """K's channels differ in size, as a model's do: a few are an order of magnitude above the rest."""
    spread = torch.randn(case["kv_heads"], case["head_dim"], generator=gen, device=dev)
    return torch.exp(0.7 * spread)


def _rows(gen, n, case, dev):
    shape = (n, case["kv_heads"], case["head_dim"])
    return torch.randn(shape, generator=gen, device=dev)


def _page_lists(case, lens, seed, dev):
    ps = case["page"]
    need = [-(-n // ps) for n in lens]
    used = sum(need)
    num_pages = used + used // 4 + 1
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed))
    indptr = [0]
    for n in need:
        indptr.append(indptr[-1] + n)
    return dict(num_pages=num_pages, page=ps,
                kv_indptr=torch.tensor(indptr, dtype=torch.int32, device=dev),
                kv_indices=perm[:used].to(torch.int32).to(dev))


def _ancestors(nodes, seed, words):
    """Visible drafted tokens of every node (itself and its ancestors) as rows of 32-bit words."""
    rng = random.Random(seed)
    rows = []
    for n in nodes:
        seen = []
        for i in range(n):
            parent = rng.randint(max(0, i - 8), i - 1) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << i))
        rows += [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for s in seen]
    return torch.tensor(rows, dtype=torch.int64)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, D, Hkv = case["op"], case["head_dim"], case["kv_heads"]
    s = dict(op=op, case=case)
    if op in ("rotary", "append8"):
        T, ps = case["tokens"], case["page"]
        num_pages = (T + T // 4) // ps + 2
        k = _rows(gen, T, case, dev) * _channels(gen, case, dev)
        s["k_new"] = k.to(torch.bfloat16)
        s["v_new"] = _rows(gen, T, case, dev).to(torch.bfloat16)
        slots = torch.randperm(num_pages * ps, generator=gen, device=dev)[:T]
        live = torch.arange(T, device=dev)
        if case["pad"]:  # padding tokens of a fixed-size batch
            off = torch.randperm(T, generator=gen, device=dev)[: case["pad"]]
            slots[off] = -1
            live = torch.nonzero(slots >= 0).flatten()
        s["slots"], s["live"] = slots, live
        shape = (num_pages, ps, Hkv, D)
        old = [torch.randn(shape, generator=gen, device=dev) for _ in range(2)]
        if op == "append8":
            (s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"]) = _quantised(old[0]), _quantised(old[1])
        else:
            s["k_pool"], s["v_pool"] = (x.to(torch.bfloat16) for x in old)
        s["interleaved"] = case["interleaved"]
        if case["rotary"]:
            R, most = case["rotary"], 4096
            s["positions"] = torch.randint(0, most, (T,), generator=gen, device=dev, dtype=torch.int32)
            freq = 1.0e6 ** (-2.0 * torch.arange(R // 2, device=dev, dtype=torch.float64) / R)
            angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
            q = torch.randn(T, case["q_heads"], D, generator=gen, device=dev)
            s["q"] = q.to(torch.bfloat16)
            s["q_out"] = torch.empty_like(s["q"])
        return s

    nodes = _nodes(case) if op == "tree" else [0] * case["batch"]
    prefix = _lengths(case, seed)
    lens = [p + n for p, n in zip(prefix, nodes)]
    s.update(_page_lists(case, lens, seed, dev))
    s["max_len"] = max(lens)
    i32 = dict(dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(lens, **i32)
    shape = (s["num_pages"], s["page"], Hkv, D)
    k = torch.randn(shape, generator=gen, device=dev) * _channels(gen, case, dev)
    v = torch.randn(shape, generator=gen, device=dev)
    if op == "tree":
        s["k_pool"], s["v_pool"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        (s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"]) = _quantised(k), _quantised(v)
    del k, v
    s["sm_scale"] = 1.0 / math.sqrt(D)
    if op == "gather8":
        # every request starts on a page of its own, so that the copy is a paged cache itself
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + -(-n // 16) * 16)
        s["out_indptr"] = torch.tensor(starts, **i32)
        s["k_out"] = torch.zeros(starts[-1], Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    N = sum(nodes) if op == "tree" else case["batch"]
    s["q"] = torch.randn(N, case["q_heads"], D, generator=gen, device=dev).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(N, case["q_heads"], dtype=torch.float32, device=dev)
    if op == "tree":
        qo = [0]
        for n in nodes:
            qo.append(qo[-1] + n)
        words = -(-max(nodes) // 32)
        s["max_nodes"] = max(nodes)
        s["qo_indptr"] = torch.tensor(qo, **i32)
        s["prefix_lens"] = torch.tensor(prefix, **i32)
        s["tree_mask"] = _ancestors(nodes, seed, words).to(torch.int32).to(dev)
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _rotated(x, cos_sin, positions, interleaved):
    """x [T, H, D] in fp32 with its first R values rotated by their positions."""
    R = cos_sin.shape[1]
    cs = cos_sin[positions.long()]
    cos, sin = cs[:, None, : R // 2], cs[:, None, R // 2:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_append(s):
    k, v = s["k_new"].float(), s["v_new"].float()
    out = {}
    if "cos_sin" in s:
        k = _rotated(k, s["cos_sin"], s["positions"], s["interleaved"])
        q = _rotated(s["q"].float(), s["cos_sin"], s["positions"], s["interleaved"])
        out["q"] = q.to(torch.bfloat16)
    live, to = s["live"], s["slots"][s["live"]]
    for name, x in (("k", k), ("v", v)):
        pool = s[name + "_pool"]
        if s["op"] == "append8":
            x8, scale = _quantised(x)
            # torch indexes no 8-bit floats: their bytes are copied
            pool.view(torch.uint8).flatten(0, 1)[to] = x8.view(torch.uint8)[live]
            s[name + "_scale"].flatten(0, 1)[to] = scale[live]
            out[name + "_scale"] = s[name + "_scale"]
        else:
            pool.flatten(0, 1)[to] = x.to(torch.bfloat16)[live]
        out[name] = pool
    return out


def _cached(s, name, slot):
    """K or V rows at the given slots in fp32."""
    pool = s[name + "_pool"].flatten(0, 1)
    if name + "_scale" not in s:
        return pool[slot].float()
    x = pool.view(torch.uint8)[slot].view(E4M3).float()
    return x * s[name + "_scale"].flatten(0, 1)[slot].unsqueeze(-1)


def _slots(s):
    """Slot of every position of every request, [B, max_len] (that of the last position behind its end), and which exist."""
    pos = torch.arange(s["max_len"], device=s["kv_lens"].device)[None, :]
    there = pos < s["kv_lens"][:, None]
    pos = torch.minimum(pos, s["kv_lens"][:, None].long() - 1)
    page = s["kv_indices"][(s["kv_indptr"][:-1, None] + pos // s["page"]).long()].long()
    return page * s["page"] + pos % s["page"], there


def _plain_gather(s):
    starts = s["out_indptr"].long()
    n = s["k_out"].shape[0]
    row = torch.arange(n, device=starts.device)
    b = torch.searchsorted(starts, row, right=True) - 1
    pos = row - starts[b]
    inside = pos < s["kv_lens"][b]
    pos = torch.where(inside, pos, 0)
    page = s["kv_indices"][(s["kv_indptr"][b] + pos // s["page"]).long()].long()
    slot = page * s["page"] + pos % s["page"]
    for name in ("k", "v"):
        got = _cached(s, name, slot).to(torch.bfloat16)
        s[name + "_out"].copy_(torch.where(inside[:, None, None], got, s[name + "_out"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _softmax_pv(score, v):
    """softmax(score) v and the log of the softmax's sum; a row without a finite score gives 0 and -inf."""
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o, (top + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    slot, there = _slots(s)
    B, Hq, D = s["q"].shape
    Hkv = s["k_pool"].shape[2]
    k = _cached(s, "k", slot).permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    score = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D), k) * s["sm_scale"]
    del k
    score = torch.where(there[:, None, None, :], score, -math.inf)
    o, lse = _softmax_pv(score, _cached(s, "v", slot).permute(0, 2, 1, 3))
    return {"out": o.reshape(B, Hq, D).to(torch.bfloat16), "lse": lse.reshape(B, Hq)}


def _plain_tree(s):
    slot, there = _slots(s)
    N, Hq, D = s["q"].shape
    Hkv = s["k_pool"].shape[2]
    B, L, M, G = slot.shape[0], s["max_len"], s["max_nodes"], Hq // Hkv
    dev = slot.device
    # rows of node m of request b, clamped to its last node where it has fewer
    qo = s["qo_indptr"].long()
    count = qo[1:] - qo[:-1]
    m = torch.arange(M, device=dev)[None, :]
    row = qo[:-1, None] + torch.minimum(m, count[:, None] - 1)
    bits = (s["tree_mask"].long()[row][..., None] >> torch.arange(32, device=dev)) & 1
    bits = bits.flatten(-2)  # [B, M, 32 * words]
    node = torch.arange(L, device=dev)[None, :] - s["prefix_lens"][:, None]  # [B, L]
    at = node.clamp(0, bits.shape[-1] - 1)[:, None, :].expand(B, M, L)
    seen = (node < 0)[:, None, :] | (torch.gather(bits, 2, at) > 0)
    seen &= there[:, None, :]
    q = s["q"].float()[row].view(B, M, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, D)
    k = _cached(s, "k", slot).permute(0, 2, 3, 1)
    score = torch.matmul(q, k) * s["sm_scale"]
    del k
    seen = seen[:, None, :, None, :].expand(B, Hkv, M, G, L).reshape(B, Hkv, M * G, L)
    score = torch.where(seen, score, -math.inf)
    o, lse = _softmax_pv(score, _cached(s, "v", slot).permute(0, 2, 1, 3))
    o = o.view(B, Hkv, M, G, D).permute(0, 2, 1, 3, 4).reshape(B, M, Hq, D)
    lse = lse.view(B, Hkv, M, G).permute(0, 2, 1, 3).reshape(B, M, Hq)
    # back to the ragged rows: row n is node n - qo[b] of its request
    n = torch.arange(N, device=dev)
    b = torch.searchsorted(qo, n, right=True) - 1
    return {"out": o[b, n - qo[b]].to(torch.bfloat16), "lse": lse[b, n - qo[b]]}


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op in ("rotary", "append8"):
        return _plain_append(s)
    return {"gather8": _plain_gather, "decode8": _plain_decode, "tree": _plain_tree}[op](s)


def _own(s):
    import paged_kv_attention_10_gb300 as pkv

    op = s["op"]
    if op == "rotary":
        pkv.rotary_kv_append(s["k_pool"], s["v_pool"], s["k_new"], s["v_new"], s["slots"], s["positions"],
                             s["cos_sin"], q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"])
        return {"k": s["k_pool"], "v": s["v_pool"], "q": s["q_out"]}
    if op == "append8":
        pool = (s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        out = {"k": pool[0], "v": pool[1], "k_scale": pool[2], "v_scale": pool[3]}
        if "cos_sin" in s:
            pkv.rotary_kv_append_fp8(*pool, s["k_new"], s["v_new"], s["slots"], s["positions"], s["cos_sin"],
                                     q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"])
            out["q"] = s["q_out"]
        else:
            pkv.kv_append_fp8(*pool, s["k_new"], s["v_new"], s["slots"])
        return out
    if op == "gather8":
        pkv.paged_gather_fp8(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["kv_indptr"],
                             s["kv_indices"], s["kv_lens"], s["out_indptr"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    c = s["case"]
    shape = (c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"])
    if "workspace" not in s:  # kept over the program's steps
        size = (pkv.tree_workspace_size(*shape, s["max_nodes"]) if op == "tree"
                else pkv.decode_fp8_workspace_size(*shape))
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    if op == "decode8":
        pkv.paged_decode_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["kv_indptr"],
                             s["kv_indices"], s["kv_lens"], s["sm_scale"], out=s["out"], lse=s["lse"],
                             workspace=s["workspace"])
    else:
        pkv.paged_tree_attention(s["q"], s["k_pool"], s["v_pool"], s["qo_indptr"], s["kv_indptr"],
                                 s["kv_indices"], s["prefix_lens"], s["tree_mask"], s["max_nodes"],
                                 s["sm_scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op, D, Hkv, Hq = case["op"], case["head_dim"], case["kv_heads"], case["q_heads"]
    row = Hkv * D
    if op in ("rotary", "append8"):
        T, live = case["tokens"], case["tokens"] - case["pad"]
        held = 2 * row if op == "rotary" else row + 4 * Hkv  # bytes of a written row of K or V
        nbytes = live * 2 * (2 * row + held) + 8 * T
        flops = 0 if op == "rotary" else 4 * live * row
        if case["rotary"]:
            nbytes += T * 2 * 2 * Hq * D + 4 * T + 4 * case["rotary"] * min(T, 4096)
            flops += 3 * case["rotary"] * (T * Hq + live * Hkv)
        return {"bytes": nbytes, "flops": flops}
    prefix = sum(_spread(case["len_min"], case["len_max"], case["batch"]))
    if op == "gather8":
        return {"bytes": prefix * 2 * (row + 4 * Hkv + 2 * row), "flops": 2 * prefix * row}
    pages = 4 * prefix // case["page"]
    if op == "decode8":
        return {"bytes": prefix * 2 * (row + 4 * Hkv) + pages + case["batch"] * Hq * (4 * D + 4),
                "flops": 4 * prefix * Hq * D}
    lens = _spread(case["len_min"], case["len_max"], case["batch"])
    nodes = _nodes(case)
    pairs = sum(n * p for n, p in zip(sorted(nodes), sorted(lens)))  # nodes' own ancestors are few
    return {"bytes": (prefix + sum(nodes)) * 4 * row + pages + sum(nodes) * Hq * (4 * D + 4),
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------
# The definition in 64 bits, request by request
# ---------------------------------------------------------------------------------------------
def _turned64(x, table, positions, interleaved):
    x = x.double().clone()
    R = table.shape[1]
    h = R // 2
    c = table.double()[positions.long(), :h].unsqueeze(1)
    sn = table.double()[positions.long(), h:].unsqueeze(1)
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, h), slice(h, R))
    z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(c, sn)
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _exact_append(s):
    out = {}
    new = {"k": s["k_new"].double(), "v": s["v_new"].double()}
    if "cos_sin" in s:
        new["k"] = _turned64(s["k_new"], s["cos_sin"], s["positions"], s["interleaved"])
        out["q"] = _turned64(s["q"], s["cos_sin"], s["positions"], s["interleaved"])
    keep = s["slots"] >= 0
    for name, x in new.items():
        held = s[name + "_pool"].double().flatten(0, 1)
        if s["op"] == "append8":
            # the values that the 8-bit ones stand for, before they are rounded to 8 bits
            mant, k = torch.frexp(x.abs().amax(-1) / 448.0)
            k = torch.where(mant == 0.5, k - 1, k)  # 2^k is amax / 448, or the next power above it
            step = ((k.long() + 1023) << 52).view(torch.float64)
            scale = s[name + "_scale"].double().flatten(0, 1)
            scale[s["slots"][keep]] = step[keep]
            out[name + "_scale"] = scale.view(s[name + "_scale"].shape)
            x = x / step.unsqueeze(-1)
        held[s["slots"][keep]] = x[keep]
        out[name] = held.view(s[name + "_pool"].shape)
    return out


def _request64(s, b, name):
    n = int(s["kv_lens"][b])
    first = int(s["kv_indptr"][b])
    pages = s["kv_indices"][first: first + -(-n // s["page"])].long()
    pool = s[name + "_pool"]
    if name + "_scale" in s:
        x = pool.view(torch.uint8)[pages].view(E4M3).double() * s[name + "_scale"][pages].double()[..., None]
    else:
        x = pool[pages].double()
    return x.flatten(0, 1)[:n].transpose(0, 1)  # [Hkv, n, D]


def _attend64(q, k, v, scale, seen=None):
    """q [Hkv, r, D] over k, v [Hkv, n, D]."""
    x = torch.bmm(q, k.transpose(1, 2)) * scale
    if seen is not None:
        x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.bmm(torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0).unsqueeze(-1)), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("rotary", "append8"):
        return _exact_append(s)
    B = case["batch"]
    if op == "gather8":
        k, v = s["k_out"].double(), s["v_out"].double()
        for b in range(B):
            at = int(s["out_indptr"][b])
            n = int(s["kv_lens"][b])
            k[at: at + n] = _request64(s, b, "k").transpose(0, 1)
            v[at: at + n] = _request64(s, b, "v").transpose(0, 1)
        return {"k": k, "v": v}
    Hkv, D = case["kv_heads"], case["head_dim"]
    G = case["q_heads"] // Hkv
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    first = s["qo_indptr"].tolist() if op == "tree" else list(range(B + 1))
    for b in range(B):
        k, v = _request64(s, b, "k"), _request64(s, b, "v")
        rows = slice(first[b], first[b + 1])
        n = first[b + 1] - first[b]
        qb = q[rows].view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        seen = None
        if op == "tree":
            seen = torch.ones(n, k.shape[1], dtype=torch.bool, device=q.device)
            p = int(s["prefix_lens"][b])
            for t in range(n):
                seen[:, p + t] = (s["tree_mask"][rows, t // 32].long() >> (t % 32)) % 2 == 1
            seen = seen.repeat_interleave(G, 0)
        o, l = _attend64(qb, k, v, s["sm_scale"], seen)
        out[rows] = o.view(Hkv, n, G, D).transpose(0, 1).reshape(n, Hkv * G, D)
        lse[rows] = l.view(Hkv, n, G).transpose(0, 1).reshape(n, Hkv * G)
    return {"out": out, "lse": lse}
