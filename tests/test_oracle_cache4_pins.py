"""The 4-bit cache's oracle against facts that do not come from it."""

import numpy as np
import pytest

from oracle import cache4


def test_e2m1_list_by_hand():
    assert cache4.E2M1_POSITIVE.tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert cache4.e2m1_values([0, 7, 8, 9, 15]).tolist() == [0.0, 6.0, 0.0, -0.5, -6.0]


def test_e2m1_rounding_by_hand():
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 100.0, 0.2, -0.2, -2.5, -2.51])
    got = cache4.e2m1_values(cache4.e2m1_codes(x))
    assert got.tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 0.0, 0.0, -2.0, -3.0]
    assert cache4.e2m1_codes(np.array([-0.1, 0.1])).tolist() == [8, 0]


def test_every_value_rounds_to_itself_and_between_neighbours_to_the_nearer():
    v = np.concatenate([-cache4.E2M1_POSITIVE[:0:-1], cache4.E2M1_POSITIVE])
    rng = np.random.default_rng(0)
    x = rng.uniform(-6, 6, 4000)
    got = cache4.e2m1_values(cache4.e2m1_codes(x))
    assert np.all(np.abs(got - x) <= np.abs(v[None, :] - x[:, None]).min(-1))
    np.testing.assert_array_equal(cache4.e2m1_values(cache4.e2m1_codes(v)), v)


def test_packing():
    codes = np.array([[1, 2, 15, 0]], dtype=np.uint8)
    assert cache4.pack(codes).tolist() == [[0x21, 0x0F]]
    np.testing.assert_array_equal(cache4.unpack(cache4.pack(codes)), codes)


@pytest.mark.parametrize("amax,g,scale", [
    (6.0, 1.0, 1.0), (6.375, 1.0, 1.0), (6.4, 1.0, 1.125), (2688.0, 1.0, 448.0), (1e9, 1.0, 448.0),
    (6 * 2.0 ** -10, 1.0, 0.0), (6 * 2.0 ** -9.9, 1.0, 2.0 ** -9), (0.0, 1.0, 0.0), (3.0, 0.5, 1.0), (12.0, 0.001, 448.0)])
def test_scales_by_hand(amax, g, scale):
    """6.375 / 6 = 1.0625 is a tie of e4m3's and goes to 1; 6 2^-10 is the tie between 0 and its smallest."""
    x = np.full((1, 16), 0.1 * amax)
    x[0, 3] = -amax
    _, s = cache4.quantise(x, g)
    assert cache4.values(np.full((1, 8), 0x22, np.uint8), s, 1.0)[0, 0] == scale


def test_a_block_by_hand():
    x = np.array([[12.0, -12.0, 1.0, 0.99, 3.0, 5.0, 7.0, 10.0, -10.01, 0.0, -0.4, 2.0, 4.0, 6.0, 8.0, 1.5]])
    packed, s = cache4.quantise(x, 1.0)  # scale 2
    want = [12, -12, 0, 0, 4, 4, 8, 8, -12, 0, 0, 2, 4, 6, 8, 2]
    # ties: 0.5 * 2 = 1 is a value of its own
    want[2] = want[3] = 1.0
    want[4] = 3.0
    got = cache4.values(packed, s, 1.0)[0]
    assert got.tolist() == [float(v) for v in want]


def test_nan_and_infinity_make_their_block_nan():
    x = np.ones((2, 32))
    x[0, 3], x[1, 31] = np.nan, -np.inf
    packed, s = cache4.quantise(x, 1.0)
    nan = np.isnan(cache4.values(packed, s, 1.0))
    want = np.zeros((2, 32), dtype=bool)
    want[0, :16] = want[1, 16:] = True
    np.testing.assert_array_equal(nan, want)
