"""fp64 reference for the 4-bit cache.

Test infrastructure only (see the package docstring).  e2m1's values are listed from the format's definition (sign, 2
exponent bits of bias 1, 1 mantissa bit) and a value is rounded by comparing it with the midpoints of that list.  The
divisions that the format's definition makes in fp32 are numpy's.
"""

from __future__ import annotations

import numpy as np

from .cache8 import E4M3_POSITIVE, e4m3_codes, e4m3_values

E2M1_POSITIVE = np.array([m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)])
_MIDPOINTS = (E2M1_POSITIVE[1:] + E2M1_POSITIVE[:-1]) / 2


def e2m1_values(codes) -> np.ndarray:
    """The values that codes (one per element) stand for."""
    codes = np.asarray(codes).astype(np.int64)
    mag = E2M1_POSITIVE[codes & 7]
    return np.where(codes & 8, -mag, mag)


def e2m1_codes(x) -> np.ndarray:
    """Codes of x rounded to the nearest e2m1 value, ties to the even code, at most 6 in size."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    lo = np.searchsorted(_MIDPOINTS, a, side="left")   # ties go down ...
    hi = np.searchsorted(_MIDPOINTS, a, side="right")  # ... or up
    code = np.where(lo % 2 == 0, lo, hi)
    return np.where(np.signbit(x), code | 8, code).astype(np.uint8)


def pack(codes) -> np.ndarray:
    """Two codes a byte, the even one in its low bits."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed) -> np.ndarray:
    packed = np.asarray(packed, dtype=np.uint8)
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def quantise(x, g):
    """(packed codes, scales as e4m3 bytes) of rows x (last axis a multiple of 16), cache scale g."""
    g = np.float32(g)
    blocks = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(blocks).all(-1)
    clean = np.where(bad[..., None], np.float32(0), blocks)
    t = np.abs(clean).max(-1) / (np.float32(6) * g)
    scale = e4m3_codes(np.minimum(t, 448.0))
    step = e4m3_values(scale).astype(np.float32) * g
    with np.errstate(over="ignore"):
        y = clean / np.where(step > 0, step, np.float32(1))[..., None]
    codes = np.where((step > 0)[..., None], e2m1_codes(np.clip(y, -8, 8)), 0)
    scale = np.where(bad, 0x7F, scale).astype(np.uint8)
    codes = np.where(bad[..., None], 0, codes)
    return pack(codes.reshape(x.shape)), scale


def values(packed, scale, g) -> np.ndarray:
    """What a cache holds, in 64 bits."""
    x = e2m1_values(unpack(packed))
    return x * np.repeat(e4m3_values(scale), 16, -1) * np.float64(np.float32(g))


__all__ = ["E2M1_POSITIVE", "E4M3_POSITIVE", "e2m1_values", "e2m1_codes", "pack", "unpack", "quantise", "values"]
