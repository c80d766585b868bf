"""Attention of one request in 64 bits with a bound on what a kernel's result may be off by.

The bound counts the kernel's roundings.  With S_j = scale sum_d |q_d k_jd| and D terms, a score in fp32
(products of exact operands, fp32 sums, a few scalings) is off by at most delta = (D + 8) 2^-24 max_j S_j;
a weight then by 2 delta (its own and the maximum's), by the exponential's 2^-21 and by its rounding
to the type the second product takes (`weight_eps`: 2^-11 f16, 2^-8 bf16), twice where the sum is not
of the rounded weights; the fp32 sums of the second product by n 2^-24.  All of these scale
A = sum_j p_j |v_j|.  The result is rounded to bf16: 2^-8 of its value.
"""

import numpy as np


def attend(q, k, v, scale, seen=None):
    """q [r, D], k and v [n, D] in fp64; seen [r, n] or None.  (o, lse, A, delta, w) with A like o,
    delta [r] and the weights w [r, n]; a row that sees nothing gives o = 0, lse = -inf."""
    x = (q @ k.T) * scale
    size = (np.abs(q) @ np.abs(k).T) * abs(scale)
    if seen is not None:
        x = np.where(seen, x, -np.inf)
        size = np.where(seen, size, 0.0)
    r = x.shape[0]
    if x.shape[1] == 0:
        z = np.zeros((r, v.shape[1]))
        return z, np.full(r, -np.inf), z, np.zeros(r), x
    top = x.max(-1)
    ok = top > -np.inf
    p = np.exp(x - np.where(ok, top, 0.0)[:, None])
    total = p.sum(-1)
    w = p / np.where(ok, total, 1.0)[:, None]
    vv = v if seen is None else np.where(seen.any(0)[:, None], v, 0.0)
    delta = (q.shape[1] + 8) * 2.0 ** -24 * size.max(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(ok, np.where(ok, top, 0.0) + np.log(np.where(ok, total, 1.0)), -np.inf)
    return w @ vv, lse, w @ np.abs(vv), delta, w


def check(out, lse, ref, n, weight_eps, what="", extra=0.0):
    """out, lse: the kernel's rows (float arrays); ref: attend()'s answer; n: positions;
    extra: what out may be off by besides."""
    o, l, A, delta, _ = ref
    tol = 2.0 ** -8 * np.abs(o) + A * (2 * weight_eps + 2 * delta[:, None] + 2.0 ** -20 + n * 2.0 ** -24) + extra
    off = np.abs(out - o)
    assert np.all(off <= tol), f"{what}: out off by {np.max(off - tol):.3g} over the bound (max {off.max():.3g})"
    if lse is not None:
        empty = np.isinf(l)
        assert np.array_equal(np.isneginf(lse), empty), f"{what}: empty rows"
        ltol = delta + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, l))
        loff = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, l))
        assert np.all(loff <= ltol), f"{what}: lse off by {np.max(loff - ltol):.3g} over the bound"
