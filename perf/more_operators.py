"""Cases for the 4-bit KV cache and for moving rows of a paged cache.

Five operators over a paged KV pool, in their plain form (elementary torch operations in 32 bits) and
as calls of the library:

  append4       quantise K/V rows to e2m1 with an e4m3 scale for every 16 values (and one scale for the whole cache)
                as they are written, with the rotation in front where the case has a rotary width
  gather4       read a 4-bit cache back as bf16 rows in position order
  decode4       one query per request over a 4-bit paged cache
  copy          copy pages, or their first rows, to other pages in every layer: a sequence forks
  compact       move the accepted tokens of drafted trees behind their prefix in every layer

``prepare`` makes the pool, page lists and new rows from the seed; ``run`` is one call; ``exact``
states the same in 64 bits.
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
        # the append of a small decode batch into a page-size-1 cache: latency alone counts
        dict(name="append4 step of 32", op="append4", tokens=32, pad=0, q_heads=0, kv_heads=8,
             head_dim=128, page=1, rotary=0, interleaved=False),
        # a long prompt's prefill in one call, an odd count with padding, neighbouring pairs over half of the head
        dict(name="append4 prefill 8191, rotary", op="append4", tokens=8191, pad=5, q_heads=32, kv_heads=8,
             head_dim=128, page=16, rotary=64, interleaved=True),
        # three short prefixes of a small model
        dict(name="gather4 3 short, D 64", op="gather4", batch=3, len_min=1, len_max=100, q_heads=0,
             kv_heads=2, head_dim=64, page=16),
        # cached prefixes of sixteen requests read back as bf16 for a prefill behind them
        dict(name="gather4 16 prefixes", op="gather4", batch=16, len_min=1, len_max=4096, q_heads=0,
             kv_heads=8, head_dim=128, page=16),
        # four short requests of a small model
        dict(name="decode4 4 short, D 64", op="decode4", batch=4, len_min=38, len_max=512, q_heads=14,
             kv_heads=2, head_dim=64, page=16),
        # a decode batch over a page-size-1 cache
        dict(name="decode4 32, page 1", op="decode4", batch=32, len_min=100, len_max=640, q_heads=16,
             kv_heads=8, head_dim=128, page=1),
        # eight long contexts: every request is split over many SMs
        dict(name="decode4 8 x 32K", op="decode4", batch=8, len_min=32768, len_max=32768, q_heads=32,
             kv_heads=8, head_dim=128, page=16),
        # the decodes of a large continuous batch
        dict(name="decode4 256, ragged", op="decode4", batch=256, len_min=512, len_max=4096, q_heads=32,
             kv_heads=8, head_dim=128, page=16),
        # four sequences fork in the middle of a page, one layer
        dict(name="copy 4 begun pages", op="copy", kind="bf16", layers=1, copies=4, partial=True,
             kv_heads=8, head_dim=128, page=16),
        # beams change places: the pages of many sequences in all layers of a model
        dict(name="copy 256 pages, 36 layers", op="copy", kind="4 bits", layers=36, copies=256, partial=False,
             kv_heads=8, head_dim=128, page=16),
        # one user's tree of eight drafted tokens, one layer of a small model
        dict(name="compact 1 x 8, D 64", op="compact", kind="bf16", layers=1, batch=1, nodes=8, taken_min=4,
             taken_max=4, len_max=100, kv_heads=2, head_dim=64, page=16),
        # a speculative step of 64 requests, trees of sixteen nodes, all layers of a model
        dict(name="compact 64 x 16, 36 layers", op="compact", kind="bf16", layers=36, batch=64, nodes=16,
             taken_min=1, taken_max=8, len_max=128, kv_heads=8, head_dim=128, page=16),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append4", "append4", "gather4", "decode4", "decode4", "decode4", "copy", "compact"])
    kv_heads, group = rng.choice([(1, 8), (2, 7), (2, 16), (3, 2), (4, 5), (4, 8), (8, 1), (8, 2), (8, 4), (16, 1)])
    head_dim = rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 16, 16, 32, 64, 24])
    base = dict(op=op, kv_heads=kv_heads, head_dim=head_dim, page=page)
    row = kv_heads * head_dim  # values of one token's K
    if op == "append4":
        tokens = _log_between(rng, 1, 8191)
        base["tokens"] = tokens
        base["pad"] = rng.choice([0, 0, tokens // 7])
        base["q_heads"] = kv_heads * group
        base["rotary"] = rng.choice([16, 32, 48, 64, head_dim])
        base["interleaved"] = rng.random() < 0.5
        if rng.random() < 0.5:
            base.update(rotary=0, interleaved=False, q_heads=0)
        return base
    if op in ("copy", "compact"):
        base["kind"] = rng.choice(["bf16", "8 bits", "4 bits"])
        base["layers"] = _log_between(rng, 1, 36)
        if op == "copy":
            # at most the bytes of the largest listed case: 256 pages of 16 tokens in 36 layers, 4.5 bits a value
            most = 256 * 16 * 36 * 1024 * 9 // 16 // (base["layers"] * page * row * 2)
            base["copies"] = _log_between(rng, 1, max(1, min(2048, most)))
            base["partial"] = rng.random() < 0.5
        else:
            most = 64 * 36 * 1024 // (base["layers"] * row)
            base["batch"] = _log_between(rng, 1, max(1, min(64, most)))
            base["nodes"] = _log_between(rng, 2, 64)
            base["taken_max"] = rng.randint(1, min(8, base["nodes"]))
            base["taken_min"] = rng.randint(0, base["taken_max"])
            base["len_max"] = _log_between(rng, 1, 128)
        return base
    base["q_heads"] = kv_heads * group
    most = 400_000 * 1024 // row  # cached tokens of one case
    longest = _log_between(rng, 1, 65536)
    base["len_max"] = longest
    base["len_min"] = max(1, longest - rng.randrange(longest))
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


# The scale of a whole cache, K's and V's: the largest value that it has seen (calibration) over 6 * 448.
GLOBAL = {"k": 0.0113, "v": 0.00235}


def _f32(x, like):
    """x rounded to fp32, on like's device: torch divides by such a tensor, and multiplies by a plain number's
    reciprocal."""
    return torch.full((), x, dtype=torch.float32, device=like.device)


def _quantised(x, cache_scale):
    """e2m1 values in fp32 and the e4m3 scale of every 16 of the last axis of x, in fp32.  The scale is the
    block's largest |x| over 6 cache_scale, a value x / (scale cache_scale), each rounded to the nearest, ties to even
    codes, and held at the type's largest."""
    g = _f32(cache_scale, x)
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    scale = (amax / (6.0 * g)).clamp(max=448.0).to(E4M3)
    step = scale.float() * g
    y = blocks / torch.where(step > 0, step, 1.0).unsqueeze(-1)
    y = torch.where(step.unsqueeze(-1) > 0, y.clamp(-6.0, 6.0), 0.0)
    # half steps below 2, whole ones below 4, steps of two above; torch rounds ties to even
    size = y.abs()
    width = torch.where(size < 2.0, 0.5, torch.where(size < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(size / width) * width, y).flatten(-2), scale


def _packed(values):
    """e2m1 values as codes, two in a byte, the even one in its low bits."""
    size = values.abs()
    code = torch.where(size < 2.0, 2.0 * size, torch.where(size < 4.0, 2.0 + size, 4.0 + size / 2.0)).to(torch.uint8)
    code |= torch.signbit(values).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _code_values(dev):
    """What the two codes of every byte stand for, as one pair of f16."""
    size = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float16, device=dev)
    value = torch.cat([size, -size])
    byte = torch.arange(256, device=dev)
    return torch.stack([value[byte & 15], value[byte >> 4]], -1)


def _channels(gen, case, dev):
    """K's channels differ in size, as a model's do: a few are an order of magnitude above the rest."""
    spread = torch.randn(case["kv_heads"], case["head_dim"], generator=gen, device=dev)
    return torch.exp(0.7 * spread)


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


def _cache4(gen, case, num_pages, dev):
    """A filled 4-bit cache: codes [2, num_pages, page, Hkv, D / 2] and scales [2, num_pages, page, Hkv, D / 16] of K and V."""
    shape = (num_pages, case["page"], case["kv_heads"], case["head_dim"])
    codes, scales = [], []
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=dev)
        if name == "k":
            x *= _channels(gen, case, dev)
        values, scale = _quantised(x, GLOBAL[name])
        codes.append(_packed(values))
        scales.append(scale)
    return torch.stack(codes), torch.stack([s.view(torch.uint8) for s in scales]).view(E4M3)


def _layers(gen, case, num_pages, dev):
    """The caches of all layers, each kind of tensor in one: [layers, 2, num_pages, page, ...] (K, then V)."""
    head = (case["layers"], 2, num_pages, case["page"], case["kv_heads"])
    D = case["head_dim"]
    if case["kind"] == "bf16":
        return [torch.randn(*head, D, generator=gen, device=dev, dtype=torch.bfloat16)]
    if case["kind"] == "8 bits":
        return [torch.randint(0, 127, (*head, D), generator=gen, device=dev, dtype=torch.uint8),
                torch.rand(head, generator=gen, device=dev)]
    return [torch.randint(0, 256, (*head, D // 2), generator=gen, device=dev, dtype=torch.uint8),
            torch.randint(0, 127, (*head, D // 16), generator=gen, device=dev, dtype=torch.uint8)]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    op, D, Hkv = case["op"], case["head_dim"], case["kv_heads"]
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(op=op, case=case)
    if op == "append4":
        T, ps = case["tokens"], case["page"]
        num_pages = T // ps + 2
        shape = (T, Hkv, D)
        k = torch.randn(shape, generator=gen, device=dev) * _channels(gen, case, dev)
        s["k_new"] = k.to(torch.bfloat16)
        s["v_new"] = torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
        slots = torch.randperm(num_pages * ps, generator=gen, device=dev)[:T]
        live = torch.arange(T, device=dev)
        if case["pad"]:  # padding tokens of a fixed-size batch
            off = torch.randperm(T, generator=gen, device=dev)[: case["pad"]]
            slots[off] = -1
            live = torch.nonzero(slots >= 0).flatten()
        s["slots"], s["live"] = slots, live
        s["codes"], s["scales"] = _cache4(gen, case, num_pages, dev)
        s["code_values"] = _code_values(dev)
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

    if op == "copy":
        n = case["copies"]
        num_pages = 2 * n + n // 8 + 1
        s["stacks"] = _layers(gen, case, num_pages, dev)
        perm = torch.randperm(num_pages, generator=gen, device=dev).int()
        s["dst"] = perm[:n].contiguous()
        # several branches of one sequence copy the same page
        s["src"] = perm[n: 2 * n][torch.randint(0, n, (n,), generator=gen, device=dev)].contiguous()
        s["rows"] = None
        if case["partial"]:
            rows = _spread(0 if n > 1 else 1, case["page"], n)
            rng.shuffle(rows)
            s["rows"] = torch.tensor(rows, **i32)
    elif op == "compact":
        B, nodes = case["batch"], case["nodes"]
        prefix = _spread(0, case["len_max"], B)
        rng.shuffle(prefix)
        s.update(_page_lists(case, [p + nodes for p in prefix], seed, dev))
        s["stacks"] = _layers(gen, case, s["num_pages"], dev)
        counts = _spread(case["taken_min"], case["taken_max"], B)
        rng.shuffle(counts)
        taken = [sorted(rng.sample(range(nodes), n)) for n in counts]
        indptr = [0]
        for t in taken:
            indptr.append(indptr[-1] + len(t))
        s["prefix_lens"] = torch.tensor(prefix, **i32)
        s["taken_indptr"] = torch.tensor(indptr, **i32)
        s["taken"] = torch.tensor([i for t in taken for i in t], **i32)
    if op in ("copy", "compact"):
        s["tensors"] = [layer[i] for stack in s["stacks"] for layer in stack for i in (0, 1)]
        return s

    lens = _lengths(case, seed)
    s.update(_page_lists(case, lens, seed, dev))
    s["max_len"] = max(lens)
    s["kv_lens"] = torch.tensor(lens, **i32)
    s["codes"], s["scales"] = _cache4(gen, case, s["num_pages"], dev)
    s["code_values"] = _code_values(dev)
    if op == "gather4":
        # every request starts on a page of its own, so that the copy is a paged cache itself
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + -(-n // 16) * 16)
        s["out_indptr"] = torch.tensor(starts, **i32)
        s["k_out"] = torch.zeros(starts[-1], Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    s["sm_scale"] = 1.0 / math.sqrt(D)
    s["q"] = torch.randn(case["batch"], case["q_heads"], D, generator=gen, device=dev).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(case["batch"], case["q_heads"], dtype=torch.float32, device=dev)
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


def _held(s, codes):
    """What the codes of a 4-bit cache stand for."""
    return torch.nn.functional.embedding(codes.int(), s["code_values"]).flatten(-2)


def _written(s):
    """The state of a 4-bit cache behind an append."""
    return {"values": _held(s, s["codes"]), "scales": s["scales"]}


def _plain_append(s):
    k, v = s["k_new"].float(), s["v_new"].float()
    out = {}
    if "cos_sin" in s:
        k = _rotated(k, s["cos_sin"], s["positions"], s["interleaved"])
        q = _rotated(s["q"].float(), s["cos_sin"], s["positions"], s["interleaved"])
        out["q"] = q.to(torch.bfloat16)
    live, to = s["live"], s["slots"][s["live"]]
    (k4, ks), (v4, vs) = _quantised(k, GLOBAL["k"]), _quantised(v, GLOBAL["v"])
    # torch indexes no 8-bit floats: their bytes are copied
    scales = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)])
    s["codes"].flatten(1, 2)[:, to] = torch.stack([_packed(k4), _packed(v4)])[:, live]
    s["scales"].view(torch.uint8).flatten(1, 2)[:, to] = scales[:, live]
    out.update(_written(s))
    return out


def _cached(s, which, slot):
    """K (0) or V (1) rows at the given slots in fp32."""
    codes = s["codes"][which].flatten(0, 1)[slot]
    scale = s["scales"].view(torch.uint8)[which].flatten(0, 1)[slot].view(E4M3).float()
    x = _held(s, codes).float().unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)
    return x.flatten(-2) * _f32(GLOBAL["kv"[which]], x)


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
    there = inside[:, None, None]
    s["k_out"].copy_(torch.where(there, _cached(s, 0, slot).to(torch.bfloat16), s["k_out"]))
    s["v_out"].copy_(torch.where(there, _cached(s, 1, slot).to(torch.bfloat16), s["v_out"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_decode(s):
    pos = torch.arange(s["max_len"], device=s["kv_lens"].device)[None, :]
    there = pos < s["kv_lens"][:, None]
    pos = torch.minimum(pos, s["kv_lens"][:, None].long() - 1)
    page = s["kv_indices"][(s["kv_indptr"][:-1, None] + pos // s["page"]).long()].long()
    slot = page * s["page"] + pos % s["page"]
    B, Hq, D = s["q"].shape
    Hkv = s["codes"].shape[3]
    k = _cached(s, 0, slot).permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    score = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D), k) * s["sm_scale"]
    del k
    score = torch.where(there[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _cached(s, 1, slot).permute(0, 2, 1, 3)) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": o.reshape(B, Hq, D).to(torch.bfloat16), "lse": lse.reshape(B, Hq)}


def _copied(s, stack):
    src, dst = s["src"].long(), s["dst"].long()
    new = stack[:, :, src]
    if s["rows"] is not None:
        keep = torch.arange(stack.shape[3], device=src.device)[None, :] < s["rows"][:, None]
        keep = keep.view(1, 1, *keep.shape, *[1] * (stack.dim() - 4))
        new = torch.where(keep, new, stack[:, :, dst])
    stack[:, :, dst] = new
    return stack


def _moved(s, stack):
    n = torch.arange(s["taken"].shape[0], device=stack.device)
    b = torch.searchsorted(s["taken_indptr"].long(), n, right=True) - 1
    first = s["prefix_lens"][b].long()
    pos = torch.stack([first + s["taken"], first + n - s["taken_indptr"][b]])  # from, to
    page = s["kv_indices"][(s["kv_indptr"][b] + pos // s["page"]).long()].long()
    slot = page * s["page"] + pos % s["page"]
    rows = stack.flatten(2, 3)
    rows[:, :, slot[1]] = rows[:, :, slot[0]]
    return stack


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op in ("copy", "compact"):
        form = _copied if op == "copy" else _moved
        return [form(s, stack) for stack in s["stacks"]]
    return {"append4": _plain_append, "gather4": _plain_gather, "decode4": _plain_decode}[op](s)


def _own(s):
    import paged_kv_attention_10_gb300 as pkv

    op = s["op"]
    if op == "copy":
        pkv.copy_pages(s["tensors"], s["src"], s["dst"], rows=s["rows"])
        return s["stacks"]
    if op == "compact":
        pkv.compact_accepted(s["tensors"], s["kv_indptr"], s["kv_indices"], s["prefix_lens"], s["taken_indptr"],
                             s["taken"])
        return s["stacks"]
    if "pool" not in s:  # the cache's tensors, which a program holds
        s["pool"] = (s["codes"][0], s["codes"][1], s["scales"][0], s["scales"][1])
    pool = s["pool"]
    scales = dict(k_global=GLOBAL["k"], v_global=GLOBAL["v"])
    if op == "append4":
        out = {}
        if "cos_sin" in s:
            pkv.rotary_kv_append_fp4(*pool, s["k_new"], s["v_new"], s["slots"], s["positions"], s["cos_sin"],
                                     q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"], **scales)
            out["q"] = s["q_out"]
        else:
            pkv.kv_append_fp4(*pool, s["k_new"], s["v_new"], s["slots"], **scales)
        out.update(_written(s))
        return out
    if op == "gather4":
        pkv.paged_gather_fp4(*pool, s["kv_indptr"], s["kv_indices"], s["kv_lens"], s["out_indptr"], s["k_out"],
                             s["v_out"], **scales)
        return {"k": s["k_out"], "v": s["v_out"]}
    if "workspace" not in s:  # kept over the program's steps
        c = s["case"]
        size = pkv.decode_fp4_workspace_size(c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"])
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    pkv.paged_decode_fp4(s["q"], *pool, s["kv_indptr"], s["kv_indices"], s["kv_lens"], s["sm_scale"], out=s["out"],
                         lse=s["lse"], workspace=s["workspace"], **scales)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _token_bytes(kind, Hkv, D):
    """Bytes of one token's K (or V) in a cache."""
    return Hkv * {"bf16": 2 * D, "8 bits": D + 4, "4 bits": D // 2 + D // 16}[kind]


def work(case):
    op, D, Hkv = case["op"], case["head_dim"], case["kv_heads"]
    row = Hkv * D
    held = _token_bytes("4 bits", Hkv, D)
    if op == "append4":
        T, live = case["tokens"], case["tokens"] - case["pad"]
        nbytes = live * 2 * (2 * row + held) + 8 * T
        flops = 4 * live * row
        if case["rotary"]:
            nbytes += T * 2 * 2 * case["q_heads"] * D + 4 * T + 4 * case["rotary"] * min(T, 4096)
            flops += 3 * case["rotary"] * (T * case["q_heads"] + live * Hkv)
        return {"bytes": nbytes, "flops": flops}
    if op in ("copy", "compact"):
        tokens = _token_bytes(case["kind"], Hkv, D) * 2 * case["layers"]
        if op == "copy":
            n = case["copies"]
            rows = _spread(0 if n > 1 else 1, case["page"], n) if case["partial"] else [case["page"]] * n
            return {"bytes": 2 * sum(rows) * tokens + 8 * n, "flops": 0}
        rows = sum(_spread(case["taken_min"], case["taken_max"], case["batch"]))
        return {"bytes": 2 * rows * tokens + 4 * rows + 16 * case["batch"], "flops": 0}
    cached = sum(_spread(case["len_min"], case["len_max"], case["batch"]))
    pages = 4 * cached // case["page"]
    if op == "gather4":
        return {"bytes": cached * 2 * (held + 2 * row) + pages, "flops": 2 * cached * row}
    return {"bytes": cached * 2 * held + pages + case["batch"] * case["q_heads"] * (4 * D + 4),
            "flops": 4 * cached * case["q_heads"] * D}


# ---------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------
def _nearest(x, values):
    """Index of the value nearest to x (ascending values), ties to the even index."""
    values = torch.tensor(values, dtype=torch.float64, device=x.device)
    between = (values[1:] + values[:-1]) / 2
    low, high = torch.bucketize(x, between), torch.bucketize(x, between, right=True)
    return torch.where(low % 2 == 0, low, high)


E2M1_SIZES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3_SIZES = [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]


def _quantised64(x, cache_scale):
    """The values that the codes stand for and the blocks' scales."""
    g = float(torch.tensor(cache_scale, dtype=torch.float32))
    sizes, scales = (torch.tensor(v, dtype=torch.float64, device=x.device) for v in (E2M1_SIZES, E4M3_SIZES))
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    scale = scales[_nearest(blocks.abs().amax(-1) / (6 * g), E4M3_SIZES)]
    size = sizes[_nearest(blocks.abs() / (scale * g).clamp(min=1e-300).unsqueeze(-1), E2M1_SIZES)]
    y = torch.where(scale.unsqueeze(-1) > 0, torch.where(blocks < 0, -size, size), 0.0)
    return y.reshape(x.shape), scale


def _rows64(codes, scales, cache_scale):
    """The rows of a 4-bit cache in 64 bits."""
    low, high = codes.long() % 16, codes.long() // 16
    pair = torch.stack([low, high], -1).flatten(-2)
    size = torch.tensor(E2M1_SIZES, dtype=torch.float64, device=codes.device)[pair % 8]
    x = torch.where(pair >= 8, -size, size)
    scale = scales.view(torch.uint8).long()  # never negative
    scale = torch.tensor(E4M3_SIZES, dtype=torch.float64, device=codes.device)[scale]
    return x * scale.repeat_interleave(16, -1) * float(torch.tensor(cache_scale, dtype=torch.float32))


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
    k, v = s["k_new"].double(), s["v_new"].double()
    if "cos_sin" in s:
        k = _turned64(s["k_new"], s["cos_sin"], s["positions"], s["interleaved"])
        out["q"] = _turned64(s["q"], s["cos_sin"], s["positions"], s["interleaved"])
    keep = s["slots"] >= 0
    to = s["slots"][keep]
    # what the other slots hold stays
    values = _rows64(s["codes"], torch.full_like(s["scales"].view(torch.uint8), 0x38), 1.0).flatten(1, 2)
    scales = s["scales"].double().flatten(1, 2)
    for i, x in enumerate((k, v)):
        y, scale = _quantised64(x, GLOBAL["kv"[i]])
        values[i][to], scales[i][to] = y[keep], scale[keep]
    out["values"] = values.view(*s["codes"].shape[:-1], -1)
    out["scales"] = scales.view(s["scales"].shape)
    return out


def _request64(s, b, which):
    n = int(s["kv_lens"][b])
    first = int(s["kv_indptr"][b])
    pages = s["kv_indices"][first: first + -(-n // s["page"])].long()
    x = _rows64(s["codes"][which][pages], s["scales"].view(torch.uint8)[which][pages], GLOBAL["kv"[which]])
    return x.flatten(0, 1)[:n].transpose(0, 1)  # [Hkv, n, D]


def exact(case, seed):
    op = case["op"]
    if op in ("copy", "compact"):
        return None  # copies: nothing is computed
    s = prepare(case, seed)
    if op == "append4":
        return _exact_append(s)
    B = case["batch"]
    if op == "gather4":
        k, v = s["k_out"].double(), s["v_out"].double()
        for b in range(B):
            at = int(s["out_indptr"][b])
            n = int(s["kv_lens"][b])
            k[at: at + n] = _request64(s, b, 0).transpose(0, 1)
            v[at: at + n] = _request64(s, b, 1).transpose(0, 1)
        return {"k": k, "v": v}
    Hkv, D, Hq = case["kv_heads"], case["head_dim"], case["q_heads"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(B):
        x = torch.bmm(q[b].view(Hkv, Hq // Hkv, D), _request64(s, b, 0).transpose(1, 2)) * s["sm_scale"]
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.bmm(torch.softmax(x, -1), _request64(s, b, 1)).reshape(Hq, D)
    return {"out": out, "lse": lse}
