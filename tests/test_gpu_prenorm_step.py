"""The operators around an FP8 Linear used together: the example's training
step against fp32, and a captured graph of every new call against eager runs
on the same inputs, replayed with eager work between."""

import importlib.util
import os

import pytest

from helpers import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def test_example_step(q):
    """Block scales leave each operand's rounding at most 2^-4 (E4M3) or 2^-3
    (E5M2) of a value; over a contraction of independent roundings the result's
    relative error is at most the operands' together: sqrt(2) 2^-4 for y, where
    both are E4M3, and sqrt(2^-8 + 2^-6) for the gradients.  dh carries the
    exact dres besides, and the norm and dgamma are sums over all of it."""
    spec = importlib.util.spec_from_file_location("prenorm_linear_step", os.path.join(ROOT, "examples", "prenorm_linear_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    err = m.run(tokens=384, K=256, N=320, micro_batches=2, seed=3)
    e4 = 2 ** 0.5 * 2.0 ** -4
    e5 = (2.0 ** -8 + 2.0 ** -6) ** 0.5
    assert err["y"] <= e4
    for name in ("dh", "dweight", "dgamma", "norm"):
        assert err[name] <= e5, (name, err)


def test_graph_of_every_call(q):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(1)
    T, C = 256, 1024
    bf = dict(device="cuda", dtype=torch.bfloat16)
    u8 = dict(device="cuda", dtype=torch.uint8)
    x, r, dy, dres = (torch.empty(T, C, **bf) for _ in range(4))
    w = torch.empty(C, **bf)
    rstd, dx = torch.empty(T, device="cuda"), torch.empty(T, C, **bf)
    dg = torch.zeros(C, device="cuda")
    big = torch.empty(70000, device="cuda")
    clipped = [torch.empty_like(dg), torch.empty_like(big)]
    plan = q.qsg_grad_plan([dg, big], clipped)
    sumsq, norm = torch.empty(1, device="cuda", dtype=torch.float64), torch.empty(1, device="cuda")
    scale, amax, three = torch.full((1,), 30.0, device="cuda"), torch.empty(1, device="cuda"), torch.empty(3, device="cuda")
    out = {k: (torch.empty(T, C, **u8), torch.empty(C, T, **u8), torch.empty(T, C, **bf)) for k in "dtmb"}
    s = {"m": (torch.empty(T, C // 32, **u8), torch.empty(C, T // 32, **u8)),
         "b": (torch.empty(T, C // 128, device="cuda"), torch.empty(C, T // 128, device="cuda"))}
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(T, C), **u8)
    cws = torch.empty(q.GRAD_WORKSPACE_BYTES, **u8)

    def fill(seed):
        gen.manual_seed(seed)
        for t in (x, r, dy, dres, w, big):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        dg.zero_()

    def step():
        for key, kind in (("d", q.DELAYED), ("t", q.TENSORWISE), ("m", q.MXFP8), ("b", q.BLOCK_1X128)):
            a, at, h = out[key]
            ss, st = s.get(key, (three if key == "t" else None, None))
            q.qsg_rmsnorm_quantize(x, w, 1e-5, kind, residual=r, h=h, rstd=rstd, q=a, qt=at, s=ss, st=st,
                                   scale=scale if key == "d" else None, amax_out=amax if key == "d" else None)
        q.qsg_rmsnorm_bwd(dy, out["d"][2], w, rstd, dx, dres=dres, dgamma=dg, accumulate=True, workspace=ws)
        q.qsg_grad_sumsq(plan, sumsq, cws)
        q.qsg_grad_clip(plan, sumsq, 1.0, norm)

    results = [*(t for k in "dtmb" for t in out[k]), *s["m"], *s["b"], rstd, dx, dg, amax, three, sumsq, norm, *clipped]
    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 6):
        fill(seed)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in results]
        for t in results:
            if t is not dg:
                t.zero_()
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, v) in enumerate(zip(results, want)):
            assert torch.equal(t, v), (seed, k)
