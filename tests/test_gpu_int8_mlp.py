"""The INT8 calls as they are used together: a training step of an MLP, part by
part against the operands that the calls themselves made, against fp32, and in
a captured graph; a decode step; other streams."""

import numpy as np
import pytest
import torch

from helpers import to_np
from oracle import int8 as o
from test_gpu_int8 import BF, F32, HALF, q, rng, same, tensor  # noqa: F401

pytestmark = pytest.mark.gpu
I8 = torch.int8


def empty(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Step:
    """y = W2 (silu(g) u), [g, u] = W1 x, and its gradients.  What is kept for
    backward is INT8: x, a and [g, u]."""

    def __init__(self, q, T, H, Fn):  # noqa: F811
        self.q, self.T, self.H, self.F = q, T, H, Fn
        r = rng(51, T, H, Fn)
        self.x, self.xf = tensor(r.standard_normal((T, H)), BF)
        self.dy, self.dyf = tensor(r.standard_normal((T, H)) * 1e-2, BF)
        self.w1, self.w1f = tensor(r.standard_normal((2 * Fn, H)) * H ** -0.5, F32)
        self.w2, self.w2f = tensor(r.standard_normal((H, Fn)) * Fn ** -0.5, F32)
        nb = -(-Fn // 128)

        def copy(n, m):
            return empty(n, m, dtype=I8), empty(n)

        self.qx, self.sx = copy(T, H)
        self.q1, self.s1 = copy(2 * Fn, H)
        self.q1t, self.s1t = copy(H, 2 * Fn)
        self.q2, self.s2 = copy(H, Fn)
        self.q2t, self.s2t = copy(Fn, H)
        self.qa, self.sa = copy(T, Fn)
        self.qdy, self.sdy = copy(T, H)
        self.qdg, self.sdg = copy(T, 2 * Fn)
        self.ck, self.cs = empty(T, 2 * Fn, dtype=I8), empty(T, 2 * nb)
        self.gu, self.dgu = empty(T, 2 * Fn, dtype=BF), empty(T, 2 * Fn, dtype=BF)
        self.da, self.y, self.dx = empty(T, Fn, dtype=BF), empty(T, H, dtype=BF), empty(T, H, dtype=BF)
        self.dw1, self.dw2 = torch.zeros(2 * Fn, H, device="cuda"), torch.zeros(H, Fn, device="cuda")
        self.ws = empty(max(q.qsg_quantize_int8_workspace(2 * Fn, H), q.qsg_quantize_int8_workspace(H, Fn)),
                        dtype=torch.uint8)

    def run(self, stream=None):
        q, k = self.q, dict(stream=stream)  # noqa: F811
        q.qsg_quantize_int8(self.w1, q=self.q1, s=self.s1, qt=self.q1t, st=self.s1t, workspace=self.ws, **k)
        q.qsg_quantize_int8(self.w2, q=self.q2, s=self.s2, qt=self.q2t, st=self.s2t, workspace=self.ws, **k)
        q.qsg_quantize_int8(self.x, q=self.qx, s=self.sx, **k)
        q.qsg_gemm_int8(self.qx, self.sx, self.q1, self.s1, self.gu, **k)
        q.qsg_swiglu_int8_store_fwd(self.gu, aq=self.qa, sa=self.sa, ck=self.ck, cs=self.cs, **k)
        q.qsg_gemm_int8(self.qa, self.sa, self.q2, self.s2, self.y, **k)
        q.qsg_quantize_int8(self.dy, q=self.qdy, s=self.sdy, **k)
        q.qsg_gemm_int8(self.qdy, self.sdy, self.q2t, self.s2t, self.da, **k)
        q.qsg_wgrad_int8(self.dy, self.qa, self.sa, self.dw2, accumulate=True, **k)
        q.qsg_swiglu_int8_store_bwd(self.da, self.ck, self.cs, self.dgu, **k)
        q.qsg_quantize_int8(self.dgu, q=self.qdg, s=self.sdg, **k)
        q.qsg_gemm_int8(self.qdg, self.sdg, self.q1t, self.s1t, self.dx, **k)
        q.qsg_wgrad_int8(self.dgu, self.qx, self.sx, self.dw1, accumulate=True, **k)

    def results(self):
        return {k: to_np(v).copy() for k, v in vars(self).items() if torch.is_tensor(v) and k != "ws"}


@pytest.mark.parametrize("T, H, Fn", [(96, 256, 384), (130, 200, 333)])
def test_training_step_part_by_part(q, T, H, Fn):  # noqa: F811
    s = Step(q, T, H, Fn)
    s.run()
    r = s.results()
    for codes, scales, x in ((r["qx"], r["sx"], s.xf), (r["q1"], r["s1"], s.w1f), (r["q1t"], r["s1t"], s.w1f.T),
                             (r["q2"], r["s2"], s.w2f), (r["q2t"], r["s2t"], s.w2f.T), (r["qdy"], r["sdy"], s.dyf),
                             (r["qdg"], r["sdg"], r["dgu"])):
        rq, rs = o.quantize(np.ascontiguousarray(x))
        assert same(codes, rq) and same(scales, rs)
    ck, cs = o.keep(r["gu"])
    assert same(r["ck"], ck) and same(r["cs"], cs)
    for c, a, b in (("gu", ("qx", "sx"), ("q1", "s1")), ("y", ("qa", "sa"), ("q2", "s2")),
                    ("da", ("qdy", "sdy"), ("q2t", "s2t")), ("dx", ("qdg", "sdg"), ("q1t", "s1t"))):
        ref = o.gemm(r[a[0]], r[a[1]], r[b[0]], r[b[1]])
        assert (np.abs(r[c] - ref) <= o.gemm_bound(ref, None, HALF[BF])).all(), c
    g, u = o.kept(ck, cs)
    _, eg, eu = o.swiglu_bounds(r["da"], g, u, HALF[BF])
    dg, du = o.swiglu_bwd(r["da"], g, u)
    assert (np.abs(r["dgu"][:, :Fn] - dg) <= eg).all() and (np.abs(r["dgu"][:, Fn:] - du) <= eu).all()
    for dw, dy, codes, scales in (("dw2", s.dyf, "qa", "sa"), ("dw1", r["dgu"], "qx", "sx")):
        ref, bound = o.wgrad(dy, r[codes], r[scales])
        assert (np.abs(r[dw] - ref) <= bound + 2.0 ** -23 * np.abs(ref)).all(), dw


def test_training_step_against_fp32(q):  # noqa: F811
    """The whole step against the MLP in fp32: 8-bit operands are off by about
    1 % of a row's largest value each, so gradients agree to a few percent of
    their norm; a missing factor or a transposed operand does not."""
    s = Step(q, 256, 256, 384)
    s.run()
    r = s.results()
    x, w1, w2, dy = (torch.from_numpy(v.copy()).double().requires_grad_() for v in (s.xf, s.w1f, s.w2f, s.dyf))
    gu = x @ w1.T
    a = torch.nn.functional.silu(gu[:, :384]) * gu[:, 384:]
    y = a @ w2.T
    y.backward(dy.detach())
    for name, ref in (("y", y), ("dx", x.grad), ("dw1", w1.grad), ("dw2", w2.grad)):
        ref = ref.detach().numpy()
        assert np.linalg.norm(r[name] - ref) < 0.05 * np.linalg.norm(ref), name


def test_training_step_in_a_graph(q):  # noqa: F811
    """Captured once, replayed on inputs changed in place, with eager steps of
    another object between: every result is the eager one, bit for bit."""
    s, e = Step(q, 130, 200, 333), Step(q, 130, 200, 333)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for replay in range(4):
        new = torch.randn(130, 200, device="cuda", generator=torch.Generator("cuda").manual_seed(replay)).to(BF)
        for k in (s, e):
            k.x.copy_(new)
            k.dw1.zero_()
            k.dw2.zero_()
        graph.replay()
        e.run()
        torch.cuda.synchronize()
        a, b = s.results(), e.results()
        for k in a:
            assert same(a[k], b[k]), (replay, k)


def test_other_streams(q):  # noqa: F811
    """Two steps at once on streams of their own, one given by its handle."""
    steps = [Step(q, 130, 200, 333) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            steps[0].run()
        steps[1].run(stream=streams[1].cuda_stream)
        steps[2].run()
    torch.cuda.synchronize()
    r = [s.results() for s in steps]
    for k in r[0]:
        assert same(r[0][k], r[2][k]) and same(r[1][k], r[2][k]), k


@pytest.mark.parametrize("rows", [1, 5, 61, 130])
def test_decode(q, rows):  # noqa: F811
    """A forward pass that keeps nothing, a batch and its tokens one by one:
    each token's result is its own, bit for bit."""
    H, Fn = 256, 400
    s = Step(q, rows, H, Fn)
    s.run()
    for n in {rows, 1}:
        for t in range(0, rows, n):
            qx, sx, qa, sa = empty(n, H, dtype=I8), empty(n), empty(n, Fn, dtype=I8), empty(n)
            gu, y = empty(n, 2 * Fn, dtype=BF), empty(n, H, dtype=BF)
            q.qsg_quantize_int8(s.x[t:t + n], q=qx, s=sx)
            q.qsg_gemm_int8(qx, sx, s.q1, s.s1, gu)
            q.qsg_swiglu_int8_store_fwd(gu, aq=qa, sa=sa)
            q.qsg_gemm_int8(qa, sa, s.q2, s.s2, y)
            assert torch.equal(gu, s.gu[t:t + n]) and torch.equal(qa, s.qa[t:t + n]) and torch.equal(y, s.y[t:t + n])
