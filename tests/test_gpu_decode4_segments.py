"""Decode over the 4-bit cache with few CTAs, so that each has segments of many stages: steps that follow one another in a
warp, stages that wrap, pages looked up from stage to stage, and two to sixteen warps that join their parts of a head."""

import numpy as np
import pytest
import torch

from test_gpu_decode4 import decode, make, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [1, 3, 8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 5])
@pytest.mark.parametrize("max_ctas,G", [(1, 2), (1, 4), (1, 5), (1, 7), (1, 12), (2, 4), (2, 7), (2, 12), (3, 4), (3, 7), (3, 12)])
def test_long_segments(lib, Hkv, G, D, page, max_ctas):
    lens = (70, 33, 200, 1, 1400, 64, 2600, 900)
    s = make(Hkv + G, lens, Hkv * G, Hkv, D, page, "any")
    out, lse, err = decode(lib, s, max_ctas=max_ctas)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("n", [65, 127, 128, 129, 191, 193, 257, 320, 385, 450, 511, 513, 577, 641, 705, 769, 833, 897, 961,
                               1023, 1025])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 64), (6, 1, 64), (2, 1, 128), (12, 2, 128), (12, 1, 64)])
def test_every_number_of_warps(lib, Hq, Hkv, D, n):
    """Segments of one stage and a little more, shared by two to all of a head's warps."""
    s = make(n, (n, 5, n - 3), Hq, Hkv, D, 16, "any")
    out, lse, err = decode(lib, s, max_ctas=1)
    assert err == 0
    verify(s, out, lse)


LAYOUTS = [(8, 2, 128, 16), (32, 8, 128, 16), (28, 4, 128, 8), (3, 1, 128, 5), (2, 1, 64, 8), (6, 1, 64, 1), (24, 2, 64, 3),
           (12, 3, 64, 32), (48, 3, 128, 16)]  # Hq, Hkv, D, page


def set_k(s, rows, scale, codes=None):
    s["scale"][0, rows] = np.asarray(scale, dtype=np.uint8).reshape(-1, 1, 1) if np.ndim(scale) else scale
    if codes is not None:
        s["codes"][0, rows] = codes
    for i, x in ((0, s["codes"]), (2, s["scale"])):
        s["pool"][i].copy_(torch.tensor(x[0]).view(s["pool"][i].shape))


@pytest.mark.parametrize("Hq,Hkv,D,page", LAYOUTS)
@pytest.mark.parametrize("at", [0, 31, 64, 700, 1999])
def test_scores_that_jump(lib, Hq, Hkv, D, page, at):
    s = make(70 + at, (2000,), Hq, Hkv, D, page)
    set_k(s, s["rows"][0][at], 0x7E)  # K of 448 times its codes
    out, lse, err = decode(lib, s, max_ctas=1)
    assert err == 0
    verify(s, out, lse, f"at {at}")


@pytest.mark.parametrize("Hq,Hkv,D,page", LAYOUTS)
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("max_ctas", [1, 2])
def test_scores_that_rise_and_fall(lib, Hq, Hkv, D, page, falling, max_ctas):
    """Every step brings a score far above (below) all of those before it."""
    n = 3000
    s = make(21, (n, 90), Hq, Hkv, D, page)
    s["q"] = s["q"].abs() + 1
    steps = 0x20 + np.arange(n) * (0x7E - 0x20) // n
    set_k(s, s["rows"][0], steps[::-1] if falling else steps, 0x77)
    out, lse, err = decode(lib, s, max_ctas=max_ctas)
    assert err == 0
    verify(s, out, lse)


@pytest.mark.parametrize("Hq,Hkv,D,page", LAYOUTS)
@pytest.mark.parametrize("at", [7, 40, 3999])
def test_nan_in_a_long_segment(lib, Hq, Hkv, D, page, at):
    s = make(9, (4000, 60), Hq, Hkv, D, page)
    G, h = Hq // Hkv, Hkv - 1
    slot = int(s["rows"][0][at])
    ks, vs = (s["pool"][i].view(-1, Hkv, D // 16) for i in (2, 3))
    held = int(vs[slot, h, 2])
    vs[slot, h, 2] = 0x7F  # V: one block of the last KV head
    out, lse, err = decode(lib, s, max_ctas=1)
    want = torch.zeros(out.shape, dtype=torch.bool)
    want[0, h * G: (h + 1) * G, 32:48] = True
    assert err == 0 and torch.equal(torch.isnan(out).cpu(), want) and not torch.isnan(lse).any()
    vs[slot, h, 2] = held
    ks[slot, 0, 1] = 0x7F  # K: all of the first KV head's queries
    out, lse, err = decode(lib, s, max_ctas=1)
    want.zero_()
    want[0, :G] = True
    assert err == 0 and torch.equal(torch.isnan(out).cpu(), want) and torch.equal(torch.isnan(lse).cpu(), want[:, :, 0])


@pytest.mark.parametrize("Hq,Hkv,D,page", LAYOUTS)
def test_a_long_segment_of_nothing_but_nan(lib, Hq, Hkv, D, page):
    s = make(19, (3000, 700), Hq, Hkv, D, page)
    set_k(s, s["rows"][0], 0x7F)
    out, lse, err = decode(lib, s, max_ctas=1)
    assert err == 0
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert not torch.isnan(out[1]).any() and not torch.isnan(lse[1]).any()


@pytest.mark.parametrize("Hq,Hkv,D,page", LAYOUTS)
def test_the_same_bits_again(lib, Hq, Hkv, D, page):
    s = make(23, (1900, 31, 4000, 77), Hq, Hkv, D, page)
    first = {n: decode(lib, s, max_ctas=n)[:2] for n in (0, 1, 5)}
    for _ in range(5):
        for n, (out, lse) in first.items():
            o, l, err = decode(lib, s, max_ctas=n)
            assert err == 0 and torch.equal(o, out) and torch.equal(l, lse)
