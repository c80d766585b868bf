"""The 8-bit cache's and the rotary append's oracle against facts that do not come from it."""

import numpy as np
import pytest
import torch

from oracle import cache8
import oracle


def test_e4m3_list_is_torchs_format():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    np.testing.assert_array_equal(cache8.e4m3_values(codes.numpy()), want)


def test_e4m3_rounding_by_hand():
    # 17 lies between 16 and 18 and ties to 16 (even mantissa); 19 between 18 and 20 ties to 20;
    # below 2^-9 / 2 everything is 0, at it the tie goes to 0, above it to 2^-9
    x = np.array([17.0, 19.0, -17.0, 2.0 ** -10, 2.0 ** -10 * 1.01, 448.0, 440.0, 0.0])
    got = cache8.e4m3_values(cache8.e4m3_codes(x))
    np.testing.assert_array_equal(got, [16.0, 20.0, -16.0, 0.0, 2.0 ** -9, 448.0, 448.0, 0.0])
    assert cache8.e4m3_codes(np.array([np.nan, np.inf, -np.inf])).tolist() == [0x7F, 0x7F, 0x7F]


def test_e4m3_rounding_against_torch():
    rng = np.random.default_rng(1)
    x = np.clip(rng.standard_normal(20000) * 2.0 ** rng.integers(-11, 8, 20000), -448, 448).astype(np.float32)
    want = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(cache8.e4m3_codes(x.astype(np.float64)), want)


@pytest.mark.parametrize("amax,k", [(448.0, 0), (449.0, 1), (1.0, -8), (1.75, -8), (1.7578125, -7),
                                    (0.0, -126), (3.0e38, 120), (1e-40, -126)])
def test_scale_by_hand(amax, k):
    x = np.array([[0.25 * amax, -amax, np.inf, np.nan]])
    assert cache8.row_scale(x)[0] == 2.0 ** k


def test_the_largest_values_stay_finite():
    codes, s = cache8.quantise(np.array([[3.3e38, -3.3895e38, 2.0 ** 127, 1.0]]))
    assert s[0] == 2.0 ** 120
    assert cache8.e4m3_values(codes)[0].tolist() == [240.0, -240.0, 128.0, 0.0]


def test_rotation_is_a_complex_product_and_agrees_with_the_half_split_oracle():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(5, 3, 32, generator=gen, dtype=torch.float64).numpy()
    pos = np.array([0, 1, 7, 1000, 31])
    ang = np.arange(1024)[:, None] * cache8.rope_frequencies(32, 1e4)
    table = np.concatenate([np.cos(ang), np.sin(ang)], -1)
    np.testing.assert_allclose(cache8.rotate(x, table, pos, False), oracle.rope(x, pos, 1e4), atol=1e-12)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * ang[pos])[:, None, :]
    got = cache8.rotate(x, table, pos, True)
    np.testing.assert_allclose(got[..., 0::2] + 1j * got[..., 1::2], z, atol=1e-12)
    part = cache8.rotate(x, table[:, [0, 1, 16, 17]], pos, False)
    np.testing.assert_array_equal(part[..., 4:], x[..., 4:])


def test_scaled_frequencies_by_hand():
    f = cache8.rope_frequencies(64, 1e4)
    np.testing.assert_array_equal(cache8.rope_frequencies(64, 1e4, "linear", 4.0), f / 4)
    turns = 8192 * f / (2 * np.pi)
    g = cache8.rope_frequencies(64, 1e4, "banded", 8.0, 8192, 1.0, 4.0)
    assert np.all(g[turns > 4] == f[turns > 4]) and np.all(g[turns < 1] == f[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((g[mid] < f[mid]) & (g[mid] > f[mid] / 8))
    # YaRN for R 64, theta 1e4, 4096 positions: dim(32) = 64 ln(4096 / (64 pi)) / (2 ln 1e4) = 10.47 -> 10,
    # dim(1) = 64 ln(4096 / (2 pi)) / (2 ln 1e4) = 22.51 -> 23
    y = cache8.rope_frequencies(64, 1e4, "yarn", 16.0, 4096, 1.0, 32.0)
    assert np.all(y[:11] == f[:11]) and np.allclose(y[23:], f[23:] / 16, rtol=1e-14)
    assert y[11] == pytest.approx(f[11] * (12 / 13 + 1 / 13 / 16), rel=1e-13)
