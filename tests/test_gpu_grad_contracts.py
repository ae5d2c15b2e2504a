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
        torch.cuda._sleep(50_000_000)  # some 20 ms
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
