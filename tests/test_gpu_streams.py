"""Calls on a stream of their own while the current stream is busy, with everything the caller may
leave out left out."""

import pytest
import torch

from test_gpu_decode8 import make as decode_step
from test_gpu_tree import make as tree_step

pytestmark = pytest.mark.gpu

BUSY = 40_000_000  # cycles, about 20 ms


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def test_tree_mask_beside_a_busy_current_stream(lib):
    n = 700
    parents, qo = i32([t - 1 for t in range(n)]), i32([0, n])
    want = lib.tree_mask_from_parents(parents, qo, n)
    assert int((want != 0).sum()) > n
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = lib.tree_mask_from_parents(parents, qo, n, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def _calls(lib):
    """name: (call on a stream, the size of its workspace); the calls make results and workspaces themselves."""
    t = tree_step(21, (3000, 31, 700), (12, 70, 3), 32, 8, 128, 16)
    tree = (t["q"], t["k"], t["v"], t["qo"], t["indptr"], t["pages"], t["prefix"])
    lens = t["prefix"] + t["qo"][1:] - t["qo"][:-1]
    d = decode_step(22, (9000, 31, 4000, 77), 32, 8, 128, 16)
    fp8 = (d["q"].cuda(), *d["pool"], d["indptr"], d["pages"], i32(d["lens"]), d["sm"])
    q = t["q"][:3].contiguous()
    # forty requests of one token over the same 3000 positions (batches above 32 have a workspace)
    pages = int(t["indptr"][1])
    count = torch.arange(41, dtype=torch.int32, device="cuda")
    many = (t["q"][:1].expand(40, -1, -1).contiguous(), t["k"], t["v"], count, count * pages, t["pages"][:pages].repeat(40),
            i32([3000] * 40))
    return {
        "tree": (lambda st: lib.paged_tree_attention(*tree, t["mask"], t["most"], t["sm"], stream=st),
                 lib.tree_workspace_size(3, 32, 8, 128, t["most"])),
        "decode8": (lambda st: lib.paged_decode_fp8(*fp8, stream=st), lib.decode_fp8_workspace_size(4, 32, 8, 128)),
        "decode": (lambda st: lib.paged_decode(q, t["k"], t["v"], t["indptr"], t["pages"], lens, t["sm"], stream=st),
                   lib.decode_workspace_size(3, 32, 8, 128)),
        "extend": (lambda st: lib.paged_extend(*many, 1, t["sm"], stream=st),
                   lib.extend_workspace_size(40, 32, 8, 128, 1)),
    }


@pytest.mark.parametrize("name", ["tree", "decode8", "decode", "extend"])
def test_workspaces_are_not_handed_on_before_the_call_is_done(lib, name):
    """Calls in a row on a side stream without a wait, while the current stream allocates and overwrites blocks of
    the sizes that the calls use.  None of the blocks that it gets is one of the calls' (each drops its
    workspace when it returns), so every result keeps its bits."""
    call, size = _calls(lib)[name]
    assert size > 0
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = call(None)
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(st):
            torch.cuda._sleep(BUSY // 200)
        got.append(call(st))
        for _ in range(3):
            torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")
            torch.full_like(want[0], float("nan"))
            torch.full_like(want[1], float("nan"))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_results_are_kept_for_the_callers_stream(lib):
    """A result of a side stream, read on the current one and dropped: the side stream's next call does not
    get its memory before the reader is done."""
    call, _ = _calls(lib)["tree"]
    st = torch.cuda.Stream()
    want = call(None)
    st.wait_stream(torch.cuda.current_stream())
    seen = []
    for _ in range(10):
        out, lse = call(st)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda._sleep(BUSY // 100)
        seen.append((out + 0, lse + 0))
        del out, lse
        with torch.cuda.stream(st):
            torch.full_like(want[0], float("nan"))
            torch.full_like(want[1], float("nan"))
    torch.cuda.synchronize()
    for out, lse in seen:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
