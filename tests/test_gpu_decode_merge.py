"""The quantised decodes' merge over partials made here: what it does with those of a decode whose CTA gave up a wait (it
reports that and leaves the result alone), which no decode can be made to do."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
SLICE = 32


@pytest.fixture(scope="module")
def merge(lib, tmp_path_factory):
    from paged_kv_attention_10_gb300 import build

    so = str(tmp_path_factory.mktemp("merge") / "merge.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", "-o", so, os.path.join(HERE, "decode_merge.cu")],
                   check=True, capture_output=True)
    return ctypes.CDLL(so).merge


class Partials:
    """Requests of `slices` slices over num_ctas CTAs of one slice each: request b's parts, and their merge in 64 bits."""

    def __init__(self, slices, seed=0):
        rng = np.random.default_rng(seed)
        B, self.ctas = len(slices), sum(slices)
        first = np.concatenate([[0], np.cumsum(slices)])[:-1] + np.arange(B)  # CTA + unit
        self.first, self.last = first, first + np.array(slices) - 1
        o = rng.standard_normal((self.ctas + B, 2, 128)).astype(np.float32)
        lse = rng.standard_normal((self.ctas + B, 2)).astype(np.float32)
        self.want, self.size = np.zeros((B, 2, 128)), np.zeros((B, 2, 128))
        self.lse = np.zeros((B, 2))
        for b in range(B):
            parts = slice(self.first[b], self.last[b] + 1)
            w = np.exp(lse[parts].astype(np.float64))
            self.lse[b] = np.log(w.sum(0))
            w = (w / w.sum(0))[..., None]
            self.want[b], self.size[b] = (w * o[parts]).sum(0), (w * np.abs(o[parts])).sum(0)
        dev = lambda x, t=torch.int32: torch.tensor(np.asarray(x), dtype=t).cuda()  # noqa: E731
        self.t = dict(lens=dev([n * SLICE for n in slices]), o=dev(o, torch.float32), lse=dev(lse, torch.float32))

    def run(self, merge, warps, first=None, last=None):
        B = len(self.first)
        dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        f, l = dev(self.first if first is None else first), dev(self.last if last is None else last)
        out = torch.full((B, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, 2), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
        assert merge(B, self.ctas, warps, p(self.t["lens"]), p(self.t["o"]), p(self.t["lse"]), p(f), p(l), p(out), p(lse),
                     p(err)) == 0
        return out.double().cpu().numpy(), lse.double().cpu().numpy(), int(err)

    def verify(self, out, lse, rows):
        # fp32 weights and sums of up to 40 terms; the result rounded to bf16
        tol = 2.0 ** -8 * np.abs(self.want) + self.size * 2.0 ** -18
        assert np.all(np.abs(out - self.want)[rows] <= tol[rows])
        assert np.all(np.abs(lse - self.lse)[rows] <= 2.0 ** -18)


SLICES = [(4,), (2, 3, 40), (2,) * 33, (3,) * 32]


@pytest.mark.parametrize("warps", [1, 8])
@pytest.mark.parametrize("slices", SLICES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_merge(merge, slices, warps):
    p = Partials(slices)
    out, lse, err = p.run(merge, warps)
    assert err == 0
    p.verify(out, lse, np.arange(len(slices)))


@pytest.mark.parametrize("warps", [1, 8])
@pytest.mark.parametrize("slices", SLICES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("end", ["first", "last"])
def test_what_a_cta_that_gave_up_leaves(merge, lib, slices, warps, end):
    """The first (last) CTA of the last request never wrote its number: the workspace holds something else there."""
    p = Partials(slices, 1)
    at = getattr(p, end).copy()
    at[-1] = -1 if end == "first" else p.ctas + len(slices)
    out, lse, err = p.run(merge, warps, **{end: at})
    assert err == lib.DEVERR_TIMEOUT
    assert np.all(out[-1] == 7) and np.all(lse[-1] == 7)
    p.verify(out, lse, np.arange(len(slices) - 1))


@pytest.mark.parametrize("B,Hq,Hkv,D,page,first", [(4, 14, 2, 64, 16, 40), (8, 32, 8, 128, 16, 900), (32, 16, 8, 128, 1, 100),
                                                   (40, 8, 1, 128, 16, 300)])
@pytest.mark.parametrize("bits", [4, 8])
def test_lengths_that_grow_between_decodes(lib, bits, B, Hq, Hkv, D, page, first):
    """Each step a kernel raises the lengths in place and the next decode starts beside it: the results are those of steps that are
    waited for one by one."""
    steps = 150
    gen = torch.Generator(device="cuda").manual_seed(B)
    need = -(-(first + steps) // page)
    head = (B * need, page, Hkv)
    u8 = lambda *s, lo=0, hi=256: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    if bits == 4:
        pool = [u8(*head, D // 2), u8(*head, D // 2), u8(*head, D // 16, lo=0x30, hi=0x48), u8(*head, D // 16, lo=0x30, hi=0x48)]
        call, size, extra = lib.paged_decode_fp4, lib.decode_fp4_workspace_size, dict(k_global=0.05, v_global=0.01)
    else:
        pool = [u8(*head, D, hi=0x40).view(torch.float8_e4m3fn) for _ in range(2)]
        pool += [torch.rand(head, device="cuda", generator=gen) + 0.5 for _ in range(2)]
        call, size, extra = lib.paged_decode_fp8, lib.decode_fp8_workspace_size, {}
    indptr = torch.arange(B + 1, dtype=torch.int32, device="cuda") * need
    pages = torch.randperm(B * need, device="cuda", generator=gen).int()
    q = torch.randn(B, Hq, D, device="cuda", generator=gen).to(torch.bfloat16)
    ws = torch.empty(size(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def run(wait):
        lens = torch.full((B,), first, dtype=torch.int32, device="cuda")
        out = torch.empty(steps, B, Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(steps, B, Hq, device="cuda")
        for t in range(steps):
            lens.add_(1)
            if wait:
                torch.cuda.synchronize()
            call(q, *pool, indptr, pages, lens, D ** -0.5, out=out[t], lse=lse[t], workspace=ws, **extra)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out, lse

    want = run(True)
    assert torch.isfinite(want[1]).all() and not torch.equal(want[0][0], want[0][-1])
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want, run(False)))
