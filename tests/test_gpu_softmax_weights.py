"""What the rounding of the softmax weights may do to a result."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from _attention64 import attend, check

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("first", [0, 5000])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (64, 1)])
def test_small_weights_behind_a_large_one_count(lib, D, page, first):
    """20000 positions whose weights are 2^-25.6 of one position's, on one SM.  They are all that some of the
    dimensions hold: 0.00039 together.

    The bound is that of _attention64 with f16 weights, 2^-11 each.  Below 2^-28 of a row's largest weight
    times value scale f16 holds a weight to 2^-39 of that instead (weights in [0, 2^15), subnormal
    below 2^-14, half a step 2^-25), the mantissa of the largest's scale counted as up to 2: 2^-38."""
    n, H = 20000, 8
    k, v = np.zeros((n, D)), np.ones((n, D))
    k[first, 0], v[first, 1:] = 16.0, 0.0
    v[:, 0] = 0.0
    v[first, 0] = 1.0
    sm = 25.6 * math.log(2.0) / 16.0
    pages = -(-n // page)
    pool = []
    for x in (k, v):
        codes, scale = cache8.quantise(x)
        assert np.array_equal(cache8.e4m3_values(codes) * scale[:, None], x)
        held, unit = np.zeros((pages * page, H, D), dtype=np.uint8), np.ones((pages * page, H), dtype=np.float32)
        held[:n], unit[:n] = codes[:, None], scale[:, None]
        pool.append((torch.tensor(held).view(pages, page, H, D).cuda(), torch.tensor(unit).view(pages, page, H).cuda()))
    q = torch.zeros(1, H, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    out, lse = lib.paged_decode_fp8(q, pool[0][0], pool[1][0], pool[0][1], pool[1][1], i32([0, pages]), i32(np.arange(pages)),
                                    i32([n]), sm, max_ctas=1)
    one = np.zeros((1, D))
    one[0, 0] = 1.0
    ref = attend(one, k, v, sm)
    extra = 2.0 ** -38 * ref[4].max() * np.abs(v).sum(0)
    for h in range(H):
        check(oracle.as_f64(out)[0, h][None], oracle.as_f64(lse)[0, h: h + 1], ref, n, 2.0 ** -11, f"head {h}", extra)


def _common_rounding(B, P, T, Hq, Hkv, D, v):
    """B requests whose position 0 has the score 0 and all others ln 0.5057: weights that bf16 holds as
    0.50390625, 0.36 % less.  v: values of all positions, [P + T, D]."""
    page, n = 16, P + T
    per = -(-n // page)
    k = torch.zeros(per * page, Hkv, D)
    k[1:, :, 0] = -1.0
    vv = torch.zeros(per * page, Hkv, D)
    vv[:n] = v[:, None]
    k, vv = (x.to(torch.bfloat16).view(per, page, Hkv, D).cuda() for x in (k, vv))
    q = torch.zeros(B * T, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    qo = i32(np.arange(B + 1) * T)
    return q, k, vv, qo, i32(np.arange(B + 1) * per), i32(np.tile(np.arange(per), B)), i32([P] * B), -math.log(0.5057)


@pytest.mark.parametrize("B,P,T,Hq,Hkv,D", [(64, 500, 4, 32, 8, 128), (64, 900, 3, 8, 8, 64), (40, 700, 60, 32, 8, 128),
                                            (1, 300, 2, 4, 4, 64)])
def test_rounding_that_the_weights_share_cancels(lib, B, P, T, Hq, Hkv, D):
    """Values that are all 1 give exactly 1, whatever the weights round to: products and their sum are off by
    fp32's n 2^-24, far less than half a step of bf16 below 1, 2^-9.  So does the extend on the same chain."""
    q, k, v, qo, indptr, pages, prefix, sm = _common_rounding(B, P, T, Hq, Hkv, D, torch.ones(P + T, D))
    mask = lib.tree_mask_from_parents(i32(np.tile(np.arange(T) - 1, B)), qo, T)
    out, _ = lib.paged_tree_attention(q, k, v, qo, indptr, pages, prefix, mask, T, sm)
    ext, _ = lib.paged_extend(q, k, v, qo, indptr, pages, prefix, T, sm)
    assert torch.all(ext == 1.0)
    assert torch.all(out == 1.0), f"{float(out.min())} to {float(out.max())}"


@pytest.mark.parametrize("B,P,T,Hq,Hkv,D", [(64, 500, 4, 32, 8, 128), (40, 700, 60, 8, 2, 64)])
def test_rounding_reaches_a_result_by_the_values_spread_only(lib, B, P, T, Hq, Hkv, D):
    """Weights p_j (1 + d_j), |d_j| <= 2^-8, over their own sum are off by sum p_j d_j (v_j - o) / sum p_j (1 + d_j):
    at most 2^-8 (1 + 2^-7) sum p_j |v_j - o|, twice that where the row is put together from parts (whose own
    results differ from o by no more on average).  The rest is _attention64's, the output's half step
    2^(e - 8) with 2^e <= |o|."""
    gen = torch.Generator().manual_seed(P)
    vals = (1.9 + 0.03 * torch.randn(P + T, D, generator=gen)).to(torch.bfloat16)
    q, k, v, qo, indptr, pages, prefix, sm = _common_rounding(B, P, T, Hq, Hkv, D, vals.float())
    mask = lib.tree_mask_from_parents(i32(np.tile(np.arange(T) - 1, B)), qo, T)
    out, lse = lib.paged_tree_attention(q, k, v, qo, indptr, pages, prefix, mask, T, sm)
    kk = np.zeros((P + T, D))
    kk[1:, 0] = -1.0
    one = np.zeros((T, D))
    one[:, 0] = 1.0
    seen = np.concatenate([np.ones((T, P), dtype=bool), np.tril(np.ones((T, T), dtype=bool))], 1)
    o, l, A, delta, w = attend(one, kk, oracle.as_f64(vals), sm, seen)
    vd = oracle.as_f64(vals)
    spread = np.stack([w[t] @ np.abs(vd - o[t]) for t in range(T)])
    tol = 2.0 ** (np.floor(np.log2(np.abs(o))) - 8) + 2 * 2.0 ** -8 * (1 + 2.0 ** -7) * spread \
        + A * (2 * delta[:, None] + 2.0 ** -20 + (P + T) * 2.0 ** -24)
    off = np.abs(oracle.as_f64(out).reshape(B, T, Hq, D) - o[None, :, None])
    assert np.all(off <= tol[None, :, None]), f"off by {off.max():.4g}, bound {tol.min():.4g}"
    ltol = delta + 2.0 ** -20 + (P + T) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l)
    assert np.all(np.abs(oracle.as_f64(lse).reshape(B, T, Hq) - l[None, :, None]) <= ltol[None, :, None])
