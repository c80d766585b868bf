"""Calls on a stream of their own while the current stream is busy, with everything the caller may
leave out left out."""

import pytest
import torch

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
