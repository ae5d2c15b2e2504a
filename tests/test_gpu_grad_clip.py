"""qsg_grad_sumsq and qsg_grad_clip against the 64-bit oracle: the sum of
squares to binary64, the norm to one binary32 rounding, the clipped values to
the roundings of the coefficient (two: the addition of 1e-6 and the division,
and the norm's own) and of the result."""

import math

import numpy as np
import pytest

import oracle
from helpers import to_np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def tensor(rng, n, dtype, std=1e-3, offset=0):
    import torch

    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((offset + n + 9,), 77.0, dtype=dt, device="cuda")
    t = buf[offset:offset + n]
    t.copy_(torch.from_numpy((rng.standard_normal(n) * std).astype(np.float32)))
    return t, buf


def call(q, plan, max_norm):
    import torch

    sumsq = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.full((q.GRAD_WORKSPACE_BYTES,), 0xFF, dtype=torch.uint8, device="cuda")
    q.qsg_grad_sumsq(plan, sumsq, ws)
    q.qsg_grad_clip(plan, sumsq, max_norm, norm)
    torch.cuda.synchronize()
    return sumsq.item(), norm.item()


def check(q, grads, max_norm, outs=None):
    values = [to_np(g).astype(np.float64) for g in grads]
    plan = q.qsg_grad_plan(grads, outs)
    sumsq, norm = call(q, plan, max_norm)
    want, s, n = oracle.norm.clip(values, max_norm)
    count = sum(v.size for v in values)
    assert abs(sumsq - s) <= s * 2.0 ** -53 * (count + 16)
    assert abs(norm - n) <= U * n * 1.001
    for g, o, v, w in zip(grads, outs or grads, values, want):
        half = 2.0 ** -8 if "bfloat16" in str(o.dtype) else U
        off = np.abs(to_np(o).astype(np.float64) - w)
        assert (off <= np.abs(w) * (half + 4 * U)).all()
        if outs is not None:
            assert np.array_equal(to_np(g).astype(np.float64), v), "the gradients are read only"


SIZES = [[1], [5], [8, 0, 3], [257, 66049, 1001], [32768], [32769, 1, 98304], [4096, 100003, 7, 70000]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("max_norm", [1e-2, 1e6])
def test_clip(q, sizes, dtype, max_norm):
    import torch

    rng = np.random.default_rng(len(sizes))
    kinds = [dtype if dtype != "mixed" else ("f32", "bf16")[k % 2] for k in range(len(sizes))]
    for offset in (0, 1, 3):
        pairs = [tensor(rng, n, k, offset=offset) for n, k in zip(sizes, kinds)]
        grads = [p[0] for p in pairs]
        # outputs whose alignment differs from the gradients'
        opairs = [tensor(rng, n, k, offset=2 * offset + 1) for n, k in zip(sizes, kinds)]
        check(q, grads, max_norm, [p[0] for p in opairs])
        check(q, grads, max_norm)
        for (t, buf), o in [(p, offset) for p in pairs] + [(p, 2 * offset + 1) for p in opairs]:
            n = t.numel()
            assert (buf[:o] == 77).all() and (buf[o + n:] == 77).all(), "written outside a tensor"


def test_shapes_and_many_tensors(q):
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    grads = [torch.randn((k % 7 + 1, 13 * (k % 11) + 1), generator=g, device="cuda") for k in range(700)]
    check(q, grads, 0.5)


def test_a_norm_below_the_limit_leaves_the_gradients(q):
    rng = np.random.default_rng(2)
    t, _ = tensor(rng, 1000, "f32")
    before = to_np(t).copy()
    call(q, q.qsg_grad_plan([t]), math.inf)
    assert np.array_equal(to_np(t), before)


@pytest.mark.parametrize("std", [1e-30, 1e25])
def test_squares_outside_binary32(q, std):
    """Squares that binary32 would lose or overflow."""
    rng = np.random.default_rng(3)
    check(q, [tensor(rng, 5000, "f32", std=std)[0]], 1.0)


def test_nothing_and_not_finite(q):
    import torch

    assert call(q, q.qsg_grad_plan([]), 1.0) == (0.0, 0.0)
    t = torch.ones(5, device="cuda")
    t[2] = float("inf")
    s, n = call(q, q.qsg_grad_plan([t]), 1.0)
    assert s == n == math.inf
    assert torch.isnan(t[2]) and (t[[0, 1, 3, 4]] == 0).all()
    t = torch.ones(5, device="cuda")
    t[2] = float("nan")
    s, n = call(q, q.qsg_grad_plan([t]), 1.0)
    assert math.isnan(s) and math.isnan(n) and torch.isnan(t).all()
    t = torch.ones(4, device="cuda")
    call(q, q.qsg_grad_plan([t]), 0.0)
    assert (t == 0).all()


def test_ranks_add_their_sums(q):
    """Two halves' sums of squares, added as an all-reduce would, clip both."""
    import torch

    rng = np.random.default_rng(5)
    a, b = tensor(rng, 40000, "f32")[0], tensor(rng, 999, "bf16")[0]
    want, s, n = oracle.norm.clip([to_np(a), to_np(b)], 1e-2)
    plans = [q.qsg_grad_plan([a]), q.qsg_grad_plan([b])]
    sums = [torch.empty(1, dtype=torch.float64, device="cuda") for _ in plans]
    ws = torch.empty(q.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for p, v in zip(plans, sums):
        q.qsg_grad_sumsq(p, v, ws)
    total = sums[0] + sums[1]
    for p in plans:
        q.qsg_grad_clip(p, total, 1e-2)
    assert (np.abs(to_np(a) - want[0]) <= np.abs(want[0]) * 6 * U).all()
    assert (np.abs(to_np(b) - want[1]) <= np.abs(want[1]) * (2.0 ** -8 + 5 * U)).all()


def test_a_tensor_of_more_than_2_31_elements(q):
    import torch

    n = (1 << 31) + 5
    t = torch.full((n,), 2.0, dtype=torch.bfloat16, device="cuda")
    s, norm = call(q, q.qsg_grad_plan([t]), 2.0 ** 9)
    assert s == 4.0 * n and norm == np.float32(math.sqrt(4.0 * n))
    k = np.float32(512.0) / (np.float32(norm) + np.float32(1e-6))
    want = torch.tensor(2.0 * float(k)).to(torch.bfloat16)
    assert t[0].item() == want.item() and torch.equal(t[-9:].cpu(), want.expand(9)) and t.min() == t.max()


def test_same_bits_twice(q):
    rng = np.random.default_rng(6)
    grads = [tensor(rng, n, "bf16")[0] for n in (300000, 5, 1234567)]
    plan = q.qsg_grad_plan(grads)
    assert call(q, plan, math.inf) == call(q, plan, math.inf)
