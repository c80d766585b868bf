"""Decode over the 4-bit cache with scores far above what a model makes: up to 2^41 in base 2.

All of a request's rows of K are alike, so their scores are the same number whatever rounding it takes, and the weights of
n positions are 1/n; or one row stands so far above the others that its weight is 1.  The result is then known without the
scores' rounding.  A weight is rounded to f16 (2^-11), the exponential is off by 2^-21 and the sums by n 2^-24, all of it
relative to A = sum_j p_j |v_j|; the result is rounded to bf16 (2^-8).  A score takes (D + 8) 2^-24 of itself (see _attention64),
the LSE a further 2^-22."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache4

pytestmark = pytest.mark.gpu

KG, VG = 0.0113, 0.00235
GROUPS = [(8, 2, 128), (7, 1, 128), (24, 2, 128), (6, 3, 64), (14, 2, 64), (12, 1, 64)]  # Hq, Hkv, D


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(seed, lens, Hq, Hkv, D, page=16):
    """K's rows are the same in all of a request; V is random."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 2
    perm = rng.permutation(num_pages)[: sum(need)]
    indptr = np.concatenate([[0], np.cumsum(need)])
    codes = np.full((2, num_pages * page, Hkv, D // 2), 0x77, dtype=np.uint8)
    scale = np.full((2, num_pages * page, Hkv, D // 16), 0x7F, dtype=np.uint8)
    rows = []
    for b, n in enumerate(lens):
        slot = perm[indptr[b] + np.arange(n) // page] * page + np.arange(n) % page
        rows.append(slot)
        codes[0, slot] = rng.integers(0, 256, (1, Hkv, D // 2)) & 0x77  # no signs
        scale[0, slot] = rng.integers(0x30, 0x40, (1, Hkv, D // 16))
        codes[1, slot], scale[1, slot] = cache4.quantise(rng.standard_normal((n, Hkv, D)), VG)
    q = (torch.tensor(rng.random((len(lens), Hq, D))) + 0.5).to(torch.bfloat16)
    return dict(codes=codes, scale=scale, rows=rows, q=q, lens=lens, num_pages=num_pages, page=page, indptr=i32(indptr),
                pages=i32(perm))


def run(lib, s, sm, max_ctas=0):
    pool = [torch.tensor(x[at].reshape(s["num_pages"], s["page"], *x.shape[2:])).cuda()
            for x in (s["codes"], s["scale"]) for at in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.paged_decode_fp4(s["q"].cuda(), *pool, s["indptr"], s["pages"], i32(s["lens"]), sm, k_global=KG, v_global=VG,
                                    err_word=err, max_ctas=max_ctas)
    assert int(err) == 0
    return oracle.as_f64(out), oracle.as_f64(lse)


def values(s, at, b):
    return cache4.values(s["codes"][at, s["rows"][b]], s["scale"][at, s["rows"][b]], (KG, VG)[at])


def scale_for(s, exponent, sign):
    """An sm_scale that takes the scores' logarithms (base 2) to 2^exponent .. 2^(exponent + 1), about."""
    k = np.abs(values(s, 0, 0)[0]).sum(-1).mean()
    return float(np.float32(sign * 2.0 ** exponent * 1.4 / (1.4427 * k)))


def verify(s, out, lse, sm, weights):
    """weights(b): of request b's positions, [n]."""
    q = oracle.as_f64(s["q"])
    Hkv, D = s["codes"].shape[2], q.shape[2]
    G = q.shape[1] // Hkv
    for b, n in enumerate(s["lens"]):
        k, v, w = values(s, 0, b), values(s, 1, b), weights(b)
        for h in range(q.shape[1]):
            want, A = w @ v[:, h // G], w @ np.abs(v[:, h // G])
            tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -10 + 2.0 ** -20 + n * 2.0 ** -24)
            assert np.all(np.abs(out[b, h] - want) <= tol), f"request {b} ({n}) head {h}: {out[b, h][:4]}, not {want[:4]}"
            x = (k[:, h // G] @ q[b, h]) * sm
            top = x.max()
            l = top + np.log(np.exp(x - top).sum())
            size = np.abs(x).max()  # all of the products have one sign
            assert abs(lse[b, h] - l) <= (D + 8) * 2.0 ** -24 * size + 2.0 ** -22 * abs(l) + 2.0 ** -19, f"lse {b} {h}"


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [0, 10, 18, 19, 20, 21, 23, 24, 25, 26, 27, 28, 29, 30, 34, 40])
@pytest.mark.parametrize("Hq,Hkv,D", GROUPS)
def test_rows_of_one_score(lib, Hq, Hkv, D, exponent, sign):
    lens = (1, 1, 2, 5, 17, 64, 65, 700) if exponent == 27 else (1, 1, 2, 65)
    s = make(exponent, lens, Hq, Hkv, D)
    sm = scale_for(s, exponent, sign)
    out, lse = run(lib, s, sm, max_ctas=1)
    verify(s, out, lse, sm, lambda b: np.full(s["lens"][b], 1 / s["lens"][b]))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [20, 27, 28, 33, 40])
@pytest.mark.parametrize("Hq,Hkv,D", GROUPS)
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_one_row_above_all_others(lib, Hq, Hkv, D, exponent, sign, max_ctas):
    """First, last and in the middle, of requests that one CTA has and of split ones."""
    lens = (2, 40, 66, 900, 4000)
    at = (1, 0, 65, 450, 3999)
    s = make(exponent + 1, lens, Hq, Hkv, D)
    for b, n in enumerate(lens):  # K of the others: half of it (of positive scores), or twice (of negative ones)
        rest = np.delete(s["rows"][b], at[b])
        s["scale"][0, rest] = s["scale"][0, rest].astype(int) + (8 if sign < 0 else -8)
    sm = scale_for(s, exponent, sign)
    out, lse = run(lib, s, sm, max_ctas)
    verify(s, out, lse, sm, lambda b: np.arange(s["lens"][b]) == at[b])


@pytest.mark.parametrize("exponent", [27, 28, 31])
@pytest.mark.parametrize("Hq,Hkv,D", GROUPS)
def test_split_rows_of_one_score(lib, Hq, Hkv, D, exponent):
    """An LSE of this size does not hold how many positions it is of, so the parts of a split request count alike: a mean
    of means, somewhere within the values."""
    s = make(exponent + 2, (5000,), Hq, Hkv, D)
    out, _ = run(lib, s, scale_for(s, exponent, 1))
    v = np.repeat(values(s, 1, 0), Hq // Hkv, 1)
    slack = np.abs(v).max() * 2.0 ** -7
    assert np.all(out[0] <= v.max(0) + slack) and np.all(out[0] >= v.min(0) - slack)
