"""Zeros in the 4-bit cache's write: the code is that of x / (scale g), whose zero has x's sign.  Bytes, no tolerance."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache4
from test_gpu_cache4 import empty, rows
from test_gpu_rotary_append import _table

pytestmark = pytest.mark.gpu


def with_zeros(seed, T, Hkv, D):
    """Zeros of both signs among a block's other values, blocks of nothing else, and values that round to zero."""
    x = rows(seed, T, Hkv, D).float().reshape(T * Hkv, D // 16, 16)
    gen = torch.Generator().manual_seed(seed)
    pick = torch.rand(x.shape, generator=gen)
    x[pick < 0.15] = -0.0
    x[pick > 0.9] = 0.0
    x[(pick > 0.4) & (pick < 0.45)] *= 2.0 ** -20
    x[::7] = -0.0
    x = x.reshape(T, Hkv, D).to(torch.bfloat16)
    assert (torch.signbit(x) & (x == 0)).any()
    return x


def held(pool, at, slots):
    return [pool[i].cpu().numpy().reshape(-1, *pool[i].shape[2:])[slots] for i in (at, 2 + at)]


@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 64), (40, 8, 128), (29, 5, 16), (31, 2, 80), (17, 1, 256)])
@pytest.mark.parametrize("g", [1.0, 0.0113])
def test_append(lib, T, Hkv, D, g):
    k, v = with_zeros(T, T, Hkv, D), with_zeros(T + 1, T, Hkv, D)
    pool = empty(T, 2, Hkv, D)
    slots = torch.randperm(2 * T, generator=torch.Generator().manual_seed(T))[:T]
    lib.kv_append_fp4(*pool, k.cuda(), v.cuda(), slots.cuda(), k_global=g, v_global=g)
    for at, x in enumerate((k, v)):
        for got, want in zip(held(pool, at, slots.numpy()), cache4.quantise(oracle.as_f64(x), g)):
            np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("Hkv,D,R,interleaved", [(8, 128, 64, True), (8, 128, 64, False), (2, 80, 48, False), (2, 80, 22, True)])
def test_rotary_append(lib, Hkv, D, R, interleaved):
    """V, and K's blocks behind the rotated ones."""
    T, g = 33, 0.0113
    k, v = with_zeros(3, T, Hkv, D), with_zeros(4, T, Hkv, D)
    pool = empty(T, 1, Hkv, D)
    pos = torch.arange(T, dtype=torch.int32)
    lib.rotary_kv_append_fp4(*pool, k.cuda(), v.cuda(), torch.arange(T).cuda(), pos.cuda(), _table(R).cuda(),
                             interleaved=interleaved, k_global=g, v_global=g)
    for got, want in zip(held(pool, 1, np.arange(T)), cache4.quantise(oracle.as_f64(v), g)):
        np.testing.assert_array_equal(got, want)
    first = -(-R // 16)
    for got, want, block in zip(held(pool, 0, np.arange(T)), cache4.quantise(oracle.as_f64(k), g), (8, 1)):
        np.testing.assert_array_equal(got[..., first * block:], want[..., first * block:])


def test_signs_come_back(lib):
    """The read-back returns the zeros as they were."""
    x = torch.full((4, 2, 64), 3.0, dtype=torch.bfloat16)
    x[..., ::3] = -0.0
    x[..., 1::3] = 0.0
    pool = empty(1, 4, 2, 64)
    lib.kv_append_fp4(*pool, x.cuda(), (-x).cuda(), torch.arange(4).cuda(), k_global=0.25, v_global=0.25)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    k, v = (torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.paged_gather_fp4(*pool, i32(0, 1), i32(0), i32(4), i32(0, 4), k, v, k_global=0.25, v_global=0.25)
    assert torch.equal(k.cpu().view(torch.int16), x.view(torch.int16))
    assert torch.equal(v.cpu().view(torch.int16), (-x).view(torch.int16))
