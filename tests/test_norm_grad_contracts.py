"""What the norm and clipping calls promise a caller who keeps a workspace, a
plan or a stream across calls, on the CPU."""

import pytest

import quantize_scaled_gemm_amd as q
from helpers import build_library, lib_is_stale


@pytest.fixture(scope="module")
def lib():
    if lib_is_stale():
        build_library()
    return q.load_library()


def test_a_workspace_serves_smaller_shapes(lib):
    """A workspace made for the longest batch and the widest row serves every
    shape with no more rows and no more columns, across the borders at which
    the kernels share their rows differently."""
    rows = [1, 2, 15, 16, 17, 63, 255, 256, 383, 384, 385, 511, 512, 513, 767, 1023, 1024, 1279, 1280, 1281, 2047, 2048,
            4096, 4097, 8192, 16383, 16384, 16385, 32768, 1 << 20]
    cols = [1, 8, 128, 255, 256, 263, 264, 519, 520, 1031, 1032, 1287, 1288, 2055, 2056, 4096, 4103, 4104, 7168, 8199,
            8200, 16384, 16391, 16392, 18439, 65536, 1 << 20, 1 << 24]
    need = {(r, c): lib.qsg_rmsnorm_bwd_workspace(r, c) for r in rows for c in cols}
    for i, r in enumerate(rows):
        for k, c in enumerate(cols):
            assert need[r, c] >= 4 * c  # a partial sum of dgamma
            if i:
                assert need[r, c] >= need[rows[i - 1], c], (r, c)
            if k:
                assert need[r, c] >= need[r, cols[k - 1]], (r, c)


def test_no_workspace_for_rows_that_the_backward_refuses(lib):
    most = 1 << 24
    assert lib.qsg_rmsnorm_bwd_workspace(4, most) > 0
    assert lib.qsg_rmsnorm_bwd_workspace(4, most + 1) == -4
    with pytest.raises(q.QsgError, match="2\\^24"):
        q.qsg_rmsnorm_bwd_workspace(0, most + 1)
