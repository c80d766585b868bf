"""Decode over the 8-bit cache with scores far above what a model makes, up to 2^41 in base 2, and V scales of many binades.

All of a request's rows of K are alike, so their scores are the same number whatever rounding it takes, and the weights of
n positions are 1/n; or one row stands so far above the others that its weight is 1.  A weight, and it times the mantissa of
V's scale, is rounded to f16 (2^-11), the exponential is off by 2^-21 and the sums by n 2^-24, all of it relative to
A = sum_j p_j |v_j|; the result is rounded to bf16 (2^-8).  A weight is held relative to the largest times V's scale (2^14), so one
below 2^-28 of that is a subnormal f16 and off by up to 2^-39 of it."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

GROUPS = [(8, 2, 128), (7, 1, 128), (24, 2, 128), (6, 3, 64), (12, 1, 64)]  # Hq, Hkv, D


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(seed, lens, Hq, Hkv, D, page, binades):
    """K's rows (no signs) are the same in all of a request; V is random, its scales 2^-binades .. 2^binades times a mantissa."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 2
    perm = rng.permutation(num_pages)[: sum(need)]
    indptr = np.concatenate([[0], np.cumsum(need)])
    codes = np.full((2, num_pages * page, Hkv, D), np.nan, dtype=np.float32)
    scale = np.full((2, num_pages * page, Hkv), np.nan, dtype=np.float32)
    rows = []
    for b, n in enumerate(lens):
        slot = perm[indptr[b] + np.arange(n) // page] * page + np.arange(n) % page
        rows.append(slot)
        codes[0, slot], scale[0, slot] = rng.integers(8, 16, (1, Hkv, D)) / 8, rng.random((1, Hkv)) + 0.5
        codes[1, slot] = rng.integers(-15, 16, (n, Hkv, D)) / 4
        scale[1, slot] = (rng.random((n, Hkv)) + 1) * 2.0 ** rng.integers(-binades, binades + 1, (n, Hkv))
    q = (torch.tensor(rng.random((len(lens), Hq, D))) + 0.5).to(torch.bfloat16)
    return dict(codes=codes, scale=scale, rows=rows, q=q, lens=lens, num_pages=num_pages, page=page, indptr=i32(indptr),
                pages=i32(perm))


def run(lib, s, sm, max_ctas):
    head = (s["num_pages"], s["page"])
    pool = [torch.tensor(x).to(torch.float8_e4m3fn).view(*head, *x.shape[1:]).cuda() for x in s["codes"]]
    pool += [torch.tensor(x).view(*head, x.shape[1]).cuda() for x in s["scale"]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = lib.paged_decode_fp8(s["q"].cuda(), *pool, s["indptr"], s["pages"], i32(s["lens"]), sm, err_word=err,
                                    max_ctas=max_ctas)
    assert int(err) == 0
    return oracle.as_f64(out), oracle.as_f64(lse)


def values(s, at, b):
    return s["codes"][at, s["rows"][b]].astype(np.float64) * s["scale"][at, s["rows"][b]][..., None]


def scale_for(s, exponent, sign):
    k = np.abs(values(s, 0, 0)[0]).sum(-1).mean()
    return float(np.float32(sign * 2.0 ** exponent * 1.4 / (1.4427 * k)))


def verify(s, out, weights):
    Hkv = s["codes"].shape[2]
    for b, n in enumerate(s["lens"]):
        v, w = values(s, 1, b), weights(b)
        for h in range(out.shape[1]):
            x = v[:, h * Hkv // out.shape[1]]
            want, A = w @ x, w @ np.abs(x)
            least = (w * s["scale"][1, s["rows"][b], h * Hkv // out.shape[1]]).max() * 2.0 ** -38
            held = np.abs(s["codes"][1, s["rows"][b], h * Hkv // out.shape[1]]).sum(0) * least
            tol = 2.0 ** -8 * np.abs(want) + A * (2.0 ** -9 + 2.0 ** -19 + n * 2.0 ** -23) + held
            assert np.all(np.abs(out[b, h] - want) <= tol), f"request {b} ({n}) head {h}: {out[b, h][:4]}, not {want[:4]}"


@pytest.mark.parametrize("binades", [0, 30])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [0, 10, 20, 22, 23, 24, 25, 26, 28, 30, 34, 40])
@pytest.mark.parametrize("Hq,Hkv,D", GROUPS)
def test_rows_of_one_score(lib, Hq, Hkv, D, exponent, sign, binades):
    s = make(exponent, (1, 1, 2, 5, 33, 200), Hq, Hkv, D, 16, binades)
    out, lse = run(lib, s, scale_for(s, exponent, sign), 1)
    verify(s, out, lambda b: np.full(s["lens"][b], 1 / s["lens"][b]))
    assert np.isfinite(lse).all()


@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [20, 24, 28, 40])
@pytest.mark.parametrize("Hq,Hkv,D", GROUPS)
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_one_row_above_all_others(lib, Hq, Hkv, D, exponent, sign, page, max_ctas):
    """First, last and in the middle, of requests that one CTA has and of split ones."""
    lens, at = (2, 40, 66, 900, 3000), (1, 0, 65, 450, 2999)
    s = make(exponent + 1, lens, Hq, Hkv, D, page, 20)
    for b, n in enumerate(lens):  # K of the others: half of it (of positive scores), or twice (of negative ones)
        s["scale"][0, np.delete(s["rows"][b], at[b])] *= 2.0 if sign < 0 else 0.5
    out, lse = run(lib, s, scale_for(s, exponent, sign), max_ctas)
    verify(s, out, lambda b: np.arange(s["lens"][b]) == at[b])
    assert np.isfinite(lse).all()
