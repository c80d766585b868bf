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
