"""The rotary append in every layout, into a bf16 and an 8-bit cache, against the fp64 oracle.

Tolerances from the arithmetic.  With the caller's fp32 table, the kernel forms x_a c - x_b s in fp32:
one product and one FMA, off by at most 2^-24 |x_b s| + 2^-24 |result| <= 2^-22 (|x_a| + |x_b|).  A bf16
result is then off by half a step, at most 2^-8 of its value; an e4m3 result by half a step, at most
2^-4 of its value, or half of the smallest step, 2^-10 scale."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from _gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _table(R, most=4096, theta=1e4):
    ang = np.arange(most)[:, None] * cache8.rope_frequencies(R, theta)
    return torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], -1), dtype=torch.float32)


def _step(seed, T, Hkv, Hq, D, R, page, pad=0, most=4096):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)  # noqa: E731
    num_pages = (T * 5 // 4) // page + 2
    slots = torch.randperm(num_pages * page, generator=gen)[:T]
    if pad:
        slots[torch.randperm(T, generator=gen)[:pad]] = -1
    return dict(k=rn(T, Hkv, D) * 3, v=rn(T, Hkv, D), q=rn(T, Hq, D) if Hq else None, slots=slots,
                pos=torch.randint(0, most, (T,), generator=gen, dtype=torch.int32), table=_table(R, most),
                k_pool=rn(num_pages, page, Hkv, D), v_pool=rn(num_pages, page, Hkv, D))


def _pair_size(x, R, interleaved):
    """|x_a| + |x_b| at every rotated value, 0 elsewhere."""
    a = np.abs(oracle.as_f64(x))
    out = np.zeros_like(a)
    if interleaved:
        s = a[..., 0:R:2] + a[..., 1:R:2]
        out[..., 0:R:2] = out[..., 1:R:2] = s
    else:
        s = a[..., : R // 2] + a[..., R // 2: R]
        out[..., : R // 2] = out[..., R // 2: R] = s
    return out


SHAPES = [
    # T, Hkv, Hq, D, R, interleaved, page, pad
    (1, 1, 1, 64, 64, False, 16, 0),
    (5, 2, 14, 64, 64, True, 16, 1),
    (131, 8, 32, 128, 128, False, 16, 17),
    (77, 3, 6, 128, 32, False, 24, 0),
    (64, 4, 4, 128, 64, True, 1, 64),
    (33, 2, 4, 80, 20, False, 8, 3),
    (33, 2, 4, 80, 22, True, 8, 3),
    (40, 1, 3, 8, 2, False, 4, 0),
    (19, 5, 5, 24, 16, False, 2, 2),
    (23, 2, 0, 256, 256, False, 16, 0),
    (23, 2, 2, 192, 96, True, 16, 0),
    (700, 16, 16, 64, 48, False, 16, 99),
]


def _ids(s):
    return "T%d-%d/%d-D%d-R%d%s-p%d" % (s[0], s[1], s[2], s[3], s[4], "i" if s[5] else "", s[6])


def _check_q(q_gpu, s, R, interleaved):
    want = cache8.rotate(s["q"], s["table"], s["pos"], interleaved)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * _pair_size(s["q"], R, interleaved)
    assert np.all(np.abs(oracle.as_f64(q_gpu) - want) <= tol)
    assert bits_equal(q_gpu[..., R:], s["q"][..., R:])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
def test_rotary_append(lib, shape, in_place):
    T, Hkv, Hq, D, R, inter, page, pad = shape
    s = _step(T + D + R, T, Hkv, Hq, D, R, page, pad)
    kp, vp = s["k_pool"].cuda(), s["v_pool"].cuda()
    q = None if s["q"] is None else s["q"].cuda()
    q_out = None if in_place or q is None else torch.full_like(q, NAN)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.rotary_kv_append(kp, vp, s["k"].cuda(), s["v"].cuda(), s["slots"].cuda(), s["pos"].cuda(),
                         s["table"].cuda(), q=q, q_out=q_out, interleaved=inter, err_word=err)
    assert int(err) == 0
    live = s["slots"] >= 0
    to = s["slots"][live]
    want = cache8.rotate(s["k"], s["table"], s["pos"], inter)[live.numpy()]
    got = kp.cpu().view(-1, Hkv, D)[to]
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * _pair_size(s["k"], R, inter)[live.numpy()]
    assert np.all(np.abs(oracle.as_f64(got) - want) <= tol)
    assert bits_equal(got[..., R:], s["k"][live][..., R:])
    v_want = s["v_pool"].clone()
    v_want.view(-1, Hkv, D)[to] = s["v"][live]
    assert bits_equal(vp, v_want)
    rest = torch.ones(kp.shape[0] * page, dtype=torch.bool)
    rest[to] = False
    assert bits_equal(kp.cpu().view(-1, Hkv, D)[rest], s["k_pool"].view(-1, Hkv, D)[rest])
    if q is not None:
        _check_q((q if in_place else q_out).cpu(), s, R, inter)
        if not in_place:
            assert bits_equal(q, s["q"])


@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
def test_rotary_append_fp8(lib, shape):
    T, Hkv, Hq, D, R, inter, page, pad = shape
    s = _step(7 * T + D + R, T, Hkv, Hq, D, R, page, pad)
    pool8 = [torch.tensor(c) for x in ("k_pool", "v_pool") for c in cache8.quantise(oracle.as_f64(s[x]))]
    k8, ks, v8, vs = [t.float().cuda() if t.dtype == torch.float64 else t.cuda() for t in pool8]
    q = None if s["q"] is None else s["q"].cuda()
    lib.rotary_kv_append_fp8(k8, v8, ks, vs, s["k"].cuda(), s["v"].cuda(), s["slots"].cuda(), s["pos"].cuda(),
                             s["table"].cuda(), q=q, interleaved=inter)
    live = (s["slots"] >= 0).numpy()
    to = s["slots"].numpy()[live]
    # V: not rotated, every byte is known
    codes, scale = cache8.quantise(oracle.as_f64(s["v"]))
    want8, want_s = pool8[2].numpy().reshape(-1, Hkv, D), pool8[3].numpy().reshape(-1, Hkv)
    want8[to], want_s[to] = codes[live], scale[live]
    np.testing.assert_array_equal(v8.cpu().numpy().reshape(-1, Hkv, D), want8)
    np.testing.assert_array_equal(vs.cpu().numpy().reshape(-1, Hkv), want_s)
    # K: the scale is the one of a row maximum within the fp32 rotation's error of the exact one
    exact = cache8.rotate(s["k"], s["table"], s["pos"], inter)[live]
    slack = 2.0 ** -22 * _pair_size(s["k"], R, inter)[live]
    got_s = ks.cpu().numpy().astype(np.float64).reshape(-1, Hkv)[to]
    big = slack.max(-1)
    amax = np.abs(exact).max(-1)
    # (scales of amax + big and amax - big, each as one row of one value)
    lo, hi = cache8.row_scale((amax - big)[..., None]), cache8.row_scale((amax + big)[..., None])
    assert np.all((got_s >= lo) & (got_s <= hi))
    got = cache8.e4m3_values(k8.cpu().numpy().reshape(-1, Hkv, D)[to]) * got_s[..., None]
    tol = 2.0 ** -4 * np.abs(exact) + 2.0 ** -10 * got_s[..., None] + 2 * slack
    assert np.all(np.abs(got - exact) <= tol)
    rest = np.ones(k8.shape[0] * page, dtype=bool)
    rest[to] = False
    np.testing.assert_array_equal(k8.cpu().numpy().reshape(-1, Hkv, D)[rest], pool8[0].numpy().reshape(-1, Hkv, D)[rest])
    np.testing.assert_array_equal(ks.cpu().numpy().reshape(-1, Hkv)[rest], pool8[1].numpy().reshape(-1, Hkv)[rest])
    if q is not None:
        _check_q(q.cpu(), s, R, inter)


def test_half_split_full_width_is_the_rope_append(lib):
    """The same layout through the older call: the same bits."""
    s = _step(3, 50, 8, 32, 128, 128, 16, 4)
    args = [s[n].cuda() for n in ("k", "v", "slots", "pos", "table")]
    a = [s["k_pool"].cuda(), s["v_pool"].cuda(), s["q"].cuda()]
    b = [x.clone() for x in a]
    lib.rope_kv_append(a[0], a[1], *args, q=a[2])
    lib.rotary_kv_append(b[0], b[1], *args, q=b[2])
    assert all(bits_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_positions_and_slots_are_skipped_and_reported(lib, fp8):
    s = _step(11, 6, 2, 4, 64, 32, 16)
    most = s["table"].shape[0]
    s["pos"][1], s["pos"][2] = most, -1
    n = s["k_pool"].shape[0] * 16
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        pool = [torch.zeros(s["k_pool"].shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        pool += [torch.zeros(s["k_pool"].shape[:3], device="cuda") for _ in range(2)]
        call = lib.rotary_kv_append_fp8
    else:
        pool = [torch.zeros_like(s["k_pool"], device="cuda") for _ in range(2)]
        call = lib.rotary_kv_append
    q_out = torch.full_like(s["q"], 7.0, device="cuda")
    args = lambda: [s[x].cuda() for x in ("k", "v", "slots", "pos", "table")]  # noqa: E731
    call(*pool, *args(), q=s["q"].cuda(), q_out=q_out, err_word=err)
    assert int(err) == lib.DEVERR_LENGTH
    written = pool[1].float().view(n, -1).abs().sum(-1).cpu() > 0
    assert sorted(torch.nonzero(written).flatten().tolist()) == sorted(s["slots"][[0, 3, 4, 5]].tolist())
    assert torch.all(q_out[1:3] == 7.0) and not torch.any(q_out[[0, 3, 4, 5]] == 7.0)
    s["pos"][1] = s["pos"][2] = 0
    s["slots"][4] = n
    err.zero_()
    call(*pool, *args(), err_word=err)
    assert int(err) == lib.DEVERR_SLOT_OOB


@pytest.mark.parametrize("kw", [
    dict(scaling="none"), dict(scaling="linear", factor=4.0),
    dict(scaling="banded", factor=8.0, original_max_position=8192),
    dict(scaling="yarn", factor=16.0, original_max_position=4096),
    dict(scaling="yarn", factor=2.5, original_max_position=1000, low=0.7, high=20.0, attention_factor=1.25)],
    ids=lambda k: k["scaling"])
@pytest.mark.parametrize("most,R,theta", [(1, 64, 1e4), (40000, 128, 1e6), (300, 20, 500.0), (5, 2, 1e4)])
def test_table(lib, most, R, theta, kw):
    t = lib.rotary_cos_sin_table(most, R, theta, **kw).cpu().double().numpy()
    yarn = kw["scaling"] == "yarn"
    f = cache8.rope_frequencies(R, theta, kw["scaling"], kw.get("factor", 1.0),
                                kw.get("original_max_position", 0.0), kw.get("low", 1.0),
                                kw.get("high", 32.0 if yarn else 4.0))
    m = kw.get("attention_factor", 0.1 * np.log(kw["factor"]) + 1.0) if yarn else 1.0
    ang = np.arange(most)[:, None] * f
    want = m * np.concatenate([np.cos(ang), np.sin(ang)], -1)
    # half an fp32 step of a value at most m, and the double angle's error: 1e5 positions * 2^-50
    assert np.abs(t - want).max() <= m * 2.0 ** -24 + 1e-9
