"""What the norm and clipping calls promise a caller who keeps a workspace, a
plan or a stream across calls, on the CPU."""

import ctypes

import pytest
import torch

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


def table(lib, entries):
    """Status of making the table of (g, out, n, dtype) entries."""
    arr = (q.Grad * len(entries))(*[q.Grad(*e, 0) for e in entries])
    n = ctypes.c_int64(0)
    assert lib.qsg_grad_plan(arr, len(entries), None, ctypes.byref(n)) == 0
    return lib.qsg_grad_plan(arr, len(entries), (q.Grad * max(1, n.value))(), ctypes.byref(n))


G, O, F = 1 << 20, 1 << 24, 1 << 28  # addresses far apart: nothing is read there


@pytest.mark.parametrize("entries", [
    [(G, G, 100, q.F32), (G, G, 100, q.F32)],              # one tensor twice, in place: it would be scaled twice
    [(G, G, 100, q.F32), (F, F, 7, q.BF16), (G, O, 100, q.F32)],
    [(G, O, 100, q.F32), (F, O, 100, q.F32)],              # one output for two gradients
    [(G, O, 100, q.F32), (F, O + 396, 100, q.F32)],        # their last and first elements
    [(G, O, 100, q.F32), (O + 8, None, 2, q.BF16)],        # an output over another gradient
    [(O + 8, None, 2, q.BF16), (G, O, 100, q.F32)],
    [(G, G + 4, 100, q.F32)],                              # an output over its own gradient, one element on
    [(G + 4, G, 100, q.F32)],
    [(G, G, 1, q.F32), (F, F, 1, q.F32), (O, O, 20000, q.F32), (O + 79996, O + 79996, 1, q.F32)],
])
def test_outputs_that_overlap_are_refused(lib, entries):
    """Chunks are clipped in any order at once: an element that two of them
    write, or that one reads and another writes, has no one value."""
    for e in (entries, entries[::-1]):
        assert table(lib, e) == -1
        assert b"overlap" in lib.qsg_last_error()


@pytest.mark.parametrize("entries", [
    [(G, G, 100, q.F32), (G + 400, G + 400, 100, q.F32), (G + 800, G + 800, 3, q.BF16)],   # slices of one buffer
    [(G, O, 100, q.F32), (G, O + 400, 100, q.F32)],        # one gradient read twice
    [(G, None, 100, q.F32), (G, None, 100, q.F32)],        # for the sum alone
    [(G, O, 100, q.F32), (G + 400, O + 400, 5, q.F32)],
    [(G, G, 0, q.F32), (G, G, 100, q.F32)],                # nothing at an address
    [(G + 400, G, 100, q.F32)],
])
def test_outputs_beside_each_other_are_taken(lib, entries):
    for e in (entries, entries[::-1]):
        assert table(lib, e) == 0, lib.qsg_last_error()


def test_the_binding_refuses_a_gradient_given_twice(lib):
    class Tensor:
        shape, dtype, device, is_cuda = (10, 10), torch.float32, "cuda:0", True

        def __init__(self, at):
            self.at = at

        def is_contiguous(self):
            return True

        def numel(self):
            return 100

        def data_ptr(self):
            return self.at

    a, b = Tensor(G), Tensor(O)
    with pytest.raises(q.QsgError, match="overlap"):
        q.qsg_grad_plan([a, b, a])


def test_a_plan_lives_for_every_stream_that_reads_it(lib, monkeypatch):
    """The table is the binding's own memory: a launch on another stream than the
    one that it was allocated on is recorded with the allocator, once per
    stream, or the memory could be given away before that launch has read it."""
    recorded = []

    class Table:
        is_cuda = True
        device = "cuda:0"

        def data_ptr(self):
            return 4096

        def record_stream(self, s):
            recorded.append(s)

    class Lib:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(q, "load_library", Lib)
    monkeypatch.setattr(q, "_stream", lambda stream: stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: (handle, device))
    plan = q.GradPlan(Table(), 1, [], [], stream=7)
    for s in (7, 9, 7, 9, 11):
        q.qsg_grad_sumsq(plan, 64, 64, stream=s)
        q.qsg_grad_clip(plan, 64, 1.0, stream=s)
    q.qsg_grad_clip(plan, 64, 1.0, stream=13)
    assert recorded == [(9, "cuda:0"), (11, "cuda:0"), (13, "cuda:0")]


def test_a_plan_on_a_raw_table(lib, monkeypatch):
    """A table that is an address, as every call here takes one, is its owner's."""
    class Lib:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(q, "load_library", Lib)
    monkeypatch.setattr(q, "_stream", lambda stream: stream)
    plan = q.GradPlan(4096, 1, [], [])
    q.qsg_grad_sumsq(plan, 64, 64, stream=9)
    q.qsg_grad_clip(plan, 64, 1.0, stream=11)
