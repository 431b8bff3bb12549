"""Sizes of the vocabulary head's loss at the edges of what one launch takes, without a GPU."""

import pytest

from w4a16_gemm_amd import head

THREADS = 512        # of a workgroup; a launch takes fewer than 2^32 threads
CHUNK = 32768        # rows taken at once at most


def rows_at_once(fn, N, K):
    """The workspace stops growing with the rows where they are taken in chunks."""
    full = fn(1 << 20, N, K, 0)
    lo, hi = 1, 1 << 20
    while lo < hi:
        mid = (lo + hi) // 2
        if fn(mid, N, K, 0) >= full:
            hi = mid
        else:
            lo = mid + 1
    return lo


@pytest.mark.parametrize("N", [8, 151936, 1 << 21, (1 << 22) - 8, 1 << 23, (1 << 24) - 8, 1 << 24])
def test_one_launch_takes_a_chunk_of_rows(N):
    lib = head._lib()
    for fn in (lib.w4a16_head_loss_workspace, lib.w4a16_head_loss_backward_workspace):
        rows = rows_at_once(fn, N, 64)
        tiles = (rows // 64 + 1) * -(-N // 256)       # the smallest tiles have 64 rows
        assert (tiles + 7) // 8 * 8 * THREADS < 1 << 32, rows
        assert fn(rows, N, 64, 0) > 0
        # workspaces are whole multiples of 256 bytes: equal ones hide a few rows at most
        if N <= 1 << 20:
            assert CHUNK - 64 <= rows <= CHUNK
