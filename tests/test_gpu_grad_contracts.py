"""What the clipping calls promise a caller who drops a plan early, leaves
outputs out or asks for the norm alone."""

import pytest

from helpers import to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def test_a_plan_dropped_while_another_stream_reads_it(q):
    """The table's memory is not given to another tensor while a launch that
    reads it waits on another stream."""
    import torch

    grads = [torch.full((5000,), 2.0, device="cuda") for _ in range(3)]
    sumsq = torch.full((1,), 60000.0, dtype=torch.float64, device="cuda")
    plan = q.qsg_grad_plan(grads)
    at, size = plan.table.data_ptr(), plan.table.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # outlasts the lines below
        q.qsg_grad_clip(plan, sumsq, 1.0)
    del plan
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    early = side.query()
    taken = any(t.data_ptr() == at for t in others)
    torch.cuda.synchronize()
    assert not early, "the launch was over before the memory was asked for"
    assert not taken
    want = 2.0 / 60000.0 ** 0.5
    for g in grads:
        assert abs(to_np(g) / want - 1).max() < 1e-6


def test_a_tensor_without_an_output_is_left_out_of_the_clip(q):
    """qsg.h lets a table for the sum alone have no outputs; a clip by such a
    table writes the others' values and the norm."""
    import ctypes

    import torch

    a, b, c = (torch.full((n,), 3.0, device="cuda") for n in (9000, 20001, 5))
    out = torch.zeros_like(c)
    entries = (q.Grad * 3)(q.Grad(a.data_ptr(), a.data_ptr(), a.numel(), q.F32, 0),
                           q.Grad(b.data_ptr(), None, b.numel(), q.F32, 0),
                           q.Grad(c.data_ptr(), out.data_ptr(), c.numel(), q.F32, 0))
    chunks, n = (q.Grad * 8)(), ctypes.c_int64(8)
    lib = q.load_library()
    assert lib.qsg_grad_plan(entries, 3, chunks, ctypes.byref(n)) == 0 and n.value == 6
    table = torch.frombuffer(chunks, dtype=torch.uint8).cuda()
    plan = q.GradPlan(table, n.value, [a, b, c], None)
    sumsq, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(q.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for max_norm in (1.0, 1e9):
        for t in (a, b, c):
            t.fill_(3.0)
        q.qsg_grad_sumsq(plan, sumsq, ws)
        q.qsg_grad_clip(plan, sumsq, max_norm, norm)
        assert sumsq.item() == 9.0 * 29006
        k = min(1.0, max_norm / (9.0 * 29006) ** 0.5)
        assert (b == 3).all() and (c == 3).all()
        assert abs(to_np(a) / (3 * k) - 1).max() < 1e-6 and abs(to_np(out) / (3 * k) - 1).max() < 1e-6


@pytest.mark.parametrize("bad", ["inf", "nan"])
@pytest.mark.parametrize("in_place", [False, True])
def test_an_infinite_limit_copies_whatever_the_norm(q, bad, in_place):
    """max_norm = infinity asks for the norm alone: one bad gradient is seen in
    the norm, and no other gradient is touched."""
    import torch

    t = torch.arange(1, 20001, device="cuda").float()
    t[777] = float(bad)
    before = to_np(t).copy()
    out = t if in_place else torch.zeros_like(t)
    sumsq, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(q.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    plan = q.qsg_grad_plan([t], [out])
    q.qsg_grad_sumsq(plan, sumsq, ws)
    q.qsg_grad_clip(plan, sumsq, float("inf"), norm)
    assert (to_np(out) == before)[[k for k in range(20000) if k != 777]].all()
    assert str(to_np(out)[777]) == bad and str(to_np(norm)[0]) == bad
