"""How much of a sum qsg_rmsnorm_bwd keeps: dgamma within the roundings that
its own rows' chains leave, whatever the number of workgroups that share them.

With u = 2^-24, a term carries the rounding of n = h rstd, and its part of
dgamma one rounding per addition of the chain that it is in: the rows that one
group of threads takes, and up to 3 additions where groups join.  The groups'
sums are added in binary64 and rounded once."""

import numpy as np
import pytest

from helpers import to_dev, to_np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def bound(rows, cols, mag, ref):
    """Groups of a full grid by the length of a row."""
    for most, groups in ((263, 8192), (519, 4096), (4103, 1024), (8199, 512), (16391, 256)):
        if cols <= most:
            break
    else:
        groups = 128
    chain = -(-rows // groups) + 3
    return U * (1 + 2.0 ** -40) * ((chain + 1) * mag + np.abs(ref))


def dgamma_of(q, dy, h, rstd, start=None):
    import torch

    rows, cols = dy.shape
    dg = to_dev(np.zeros(cols, np.float32) if start is None else start)
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dx = torch.empty(dy.shape, device="cuda")
    q.qsg_rmsnorm_bwd(to_dev(dy), to_dev(h), torch.ones(cols, device="cuda"), to_dev(rstd), dx, dgamma=dg,
                      accumulate=start is not None, workspace=ws)
    return to_np(dg).astype(np.float64)


SHAPES = [(1, 5), (333, 40), (333, 1111), (383, 4096), (300, 8192), (250, 16384), (120, 16400), (1200, 2049),
          (8000, 24), (4000, 500), (9000, 40), (5000, 300), (2500, 1111), (1200, 4104), (600, 9000)]


@pytest.mark.parametrize("rows, cols", SHAPES)
def test_small_terms_beside_a_large_one(q, rows, cols):
    """One row of 2^24 and the rest of 2^-4 each: a chain of binary32 additions
    from the large one on keeps none of them."""
    dy = np.full((rows, cols), 2.0 ** -4, np.float32)
    dy[rows // 3] = 2.0 ** 24
    ref = dy.astype(np.float64).sum(axis=0)
    for start in (None, np.full(cols, 2.0 ** -5, np.float32)):
        got = dgamma_of(q, dy, np.ones_like(dy), np.ones(rows, np.float32), start)
        want = ref + (0 if start is None else start)
        assert (np.abs(got - want) <= bound(rows, cols, want, want)).all(), np.abs(got - want).max()


@pytest.mark.parametrize("rows, cols", SHAPES)
def test_random_terms(q, rows, cols):
    rng = np.random.default_rng([rows, cols])
    dy = rng.standard_normal((rows, cols)).astype(np.float32)
    h = rng.standard_normal((rows, cols)).astype(np.float32)
    rstd = rng.uniform(0.5, 2, rows).astype(np.float32)
    term = dy.astype(np.float64) * h * rstd[:, None].astype(np.float64)
    got = dgamma_of(q, dy, h, rstd)
    ref, mag = term.sum(axis=0), np.abs(term).sum(axis=0)
    assert (np.abs(got - ref) <= bound(rows, cols, mag, ref)).all()
