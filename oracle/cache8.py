"""fp64 reference for the rotary append in every layout and for the 8-bit cache.

Test infrastructure only (see the package docstring).  The e4m3 values are listed from the format's
definition (sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities, 0x7f and 0xff NaN) and a
value is rounded by comparing it with the midpoints of that list, so nothing here shares a
conversion with the code it checks.
"""

from __future__ import annotations

import numpy as np

from .attention import _as_int, as_f64


def _e4m3_positive():
    v = []
    for code in range(127):  # 0x00 .. 0x7e
        e, m = divmod(code, 8)
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3_POSITIVE = _e4m3_positive()  # ascending, 0 .. 448
_MIDPOINTS = (E4M3_POSITIVE[1:] + E4M3_POSITIVE[:-1]) / 2


def e4m3_values(codes) -> np.ndarray:
    """The values that e4m3 bytes stand for."""
    codes = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    mag = np.append(E4M3_POSITIVE, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def e4m3_codes(x) -> np.ndarray:
    """Bytes of x rounded to the nearest e4m3 value, ties to the even code; |x| <= 448 or not finite
    (NaN without regard to its sign bit: 0x7f)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert a.max(initial=0.0) <= 448.0
    lo = np.searchsorted(_MIDPOINTS, a, side="left")   # ties go down ...
    hi = np.searchsorted(_MIDPOINTS, a, side="right")  # ... or up
    code = np.where(lo % 2 == 0, lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def row_scale(x) -> np.ndarray:
    """The power-of-two scale of every row (last axis): the smallest 2^k, k >= -126, with the
    largest finite |x| at most 448 * 2^k."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=-1)
    k = np.full(a.shape, -126)
    for _ in range(2 * 126 + 4):  # count up: no logarithm to round
        k = np.where(a > 448.0 * 2.0 ** k.astype(np.float64), k + 1, k)
    return 2.0 ** k.astype(np.float64)


def quantise(x):
    """(bytes, scales) of rows x (any leading shape, fp64)."""
    x = np.asarray(x, dtype=np.float64)
    s = row_scale(x)
    y = x / s[..., None]
    # at the largest scale 256 would stand for 2^128: the largest value below it is held instead
    top = (s[..., None] == 2.0 ** 120) & np.isfinite(y)
    return e4m3_codes(np.where(top, np.clip(np.where(top, y, 0.0), -240.0, 240.0), y)), s


def rotate(x, cos_sin, positions, interleaved):
    """x [T, H, D] with its first R values rotated; cos_sin [max_position, R] as the caller gives it."""
    x = as_f64(x).copy()
    t = as_f64(cos_sin)[_as_int(positions)]
    R = t.shape[1]
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = t[:, i, None], t[:, R // 2 + i, None]
        xa, xb = x[:, :, a].copy(), x[:, :, b].copy()
        x[:, :, a] = xa * c - xb * s
        x[:, :, b] = xb * c + xa * s
    return x


def rope_frequencies(R, theta, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """The R / 2 frequencies theta^(-2i/R), scaled for long contexts."""
    i = np.arange(R // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / R)
    if scaling == "none":
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "banded":
        wavelength = 2 * np.pi / f
        s = (original / wavelength - low) / (high - low)
        return np.where(s >= 1, f, np.where(s <= 0, f / factor, (1 - s) * f / factor + s * f))
    assert scaling == "yarn"
    dim = lambda turns: R * np.log(original / (turns * 2 * np.pi)) / (2 * np.log(theta))  # noqa: E731
    lo, hi = max(np.floor(dim(high)), 0), min(np.ceil(dim(low)), R - 1)
    if lo == hi:
        hi += 0.001
    extrapolated = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    return f / factor * (1 - extrapolated) + f * extrapolated
