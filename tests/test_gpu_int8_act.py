"""The gated activation that keeps its input in INT8: codes and scales
bit-exact, values within the roundings of their binary32 evaluation, the
gradient against the formula's and against differences."""

import numpy as np
import pytest
import torch

from helpers import to_np
from oracle import int8 as o
from test_gpu_int8 import BF, F32, HALF, q, rng, same, same_scales, tensor  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (2, 127), (5, 128), (4, 129), (300, 16), (7, 250), (16, 256), (3, 1111), (2, 2048),
          (2, 2049), (3, 4096), (2, 8192), (2, 8200), (1, 14336), (2, 16384), (1, 16385), (2, 32768), (1, 32769),
          (2, 33001), (1200, 130)]


def make(q, gu, cols, **outs):
    R, dt = gu.shape[0], gu.dtype
    nb = -(-cols // 128)
    all_outs = dict(a=((R, cols), dt), aq=((R, cols), torch.int8), sa=((R,), F32), ck=((R, 2 * cols), torch.int8),
                    cs=((R, 2 * nb), F32))
    made = {k: torch.full(*all_outs[k][:1], 99, dtype=all_outs[k][1], device="cuda") for k in outs if outs[k]}
    q.qsg_swiglu_int8_store_fwd(gu, **made)
    return {k: to_np(v) for k, v in made.items()}


def check_forward(got, gu, dtype):
    C = gu.shape[1] // 2
    g, u = gu[:, :C], gu[:, C:]
    ref = o.swiglu(g, u)
    if "ck" in got:
        rq, rs = o.keep(gu)
        assert same_scales(got["cs"], rs)
        assert same(got["ck"], rq)
    if "a" in got:
        bound = o.swiglu_bounds(None, g, u, HALF[dtype])[0]
        bad = ~(np.abs(got["a"] - ref) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    if "aq" in got:
        # the scale carries the error of the row's maximum and its own rounding;
        # a code is off by half a step, and by what its value and the scale are off
        ea = o.swiglu_bounds(None, g, u, 0.0)[0]
        top = np.abs(ref).max(axis=1, initial=0)
        at = ea.max(axis=1, initial=0)
        want = np.where(top == 0, 1, np.maximum(top / 127, 2.0 ** -126))
        assert (np.abs(got["sa"] - want) <= at / 127 + 2.0 ** -23 * want).all()
        s = got["sa"].astype(np.float64)[:, None]
        assert (np.abs(got["aq"].astype(np.float64) * s - ref) <= s * (0.5 + 127 * 2.0 ** -22) + ea).all()
        assert (np.abs(got["aq"].astype(np.int64)) <= 127).all()
        assert all(np.abs(r).max(initial=0) == 127 for r, t in zip(got["aq"].astype(np.int64), top) if t > 1e-30)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R, C", SHAPES)
def test_forward(q, R, C, dtype):  # noqa: F811
    gd, gf = tensor(rng(21, R, C).standard_normal((R, 2 * C)) * 4, dtype)
    check_forward(make(q, gd, C, a=1, ck=1, cs=1), gf, dtype)
    check_forward(make(q, gd, C, a=1, aq=1, sa=1, ck=1, cs=1), gf, dtype)


@pytest.mark.parametrize("outs", [("a",), ("ck", "cs"), ("aq", "sa"), ("aq", "sa", "a"), ("aq", "sa", "ck", "cs")],
                         ids="+".join)
@pytest.mark.parametrize("C", [136, 40000])
def test_outputs_one_by_one(q, outs, C):  # noqa: F811
    gd, gf = tensor(rng(22, C).standard_normal((3, 2 * C)) * 3, BF)
    check_forward(make(q, gd, C, **dict.fromkeys(outs, 1)), gf, BF)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_forward_extremes(q, dtype):  # noqa: F811
    """Gates far on either side, where the exponential overflows or vanishes."""
    C = 300
    g = np.concatenate([np.linspace(-120, 120, 2 * C - 4), [0, -0.0, 1e-30, -1e-30]]).reshape(2, C)
    gd, gf = tensor(np.concatenate([g, rng(23).standard_normal((2, C))], axis=1), dtype)
    check_forward(make(q, gd, C, a=1, ck=1, cs=1), gf, dtype)


def test_not_finite(q):  # noqa: F811
    """A block with an infinity or a NaN keeps NaN scales and codes of 0, its
    neighbours their own; the row's INT8 copy of a has a NaN scale."""
    C = 300
    x = rng(24).standard_normal((4, 2 * C)).astype(np.float32)
    x[1, 130], x[2, C + 299], x[3, 0] = np.inf, np.nan, -np.inf
    gd, gf = tensor(x, BF)
    for outs in (dict(ck=1, cs=1), dict(ck=1, cs=1, aq=1, sa=1)):
        got = make(q, gd, C, **outs)
        rq, rs = o.keep(gf)
        assert same_scales(got["cs"], rs) and same(got["ck"], rq)
        assert np.isnan(rs).sum() == 3
        if "aq" in got:
            assert np.isnan(got["sa"][1:]).all() and not got["aq"][1:].any() and np.isfinite(got["sa"][0])


def backward(q, da, ck, cs, again, pad=0):
    R, C = da.shape
    full = torch.full((R, 2 * C + pad), 7.0, dtype=da.dtype, device="cuda")
    a = torch.full((R, C), 99.0, dtype=da.dtype, device="cuda") if again else None
    q.qsg_swiglu_int8_store_bwd(da, torch.from_numpy(ck).cuda(), torch.from_numpy(cs).cuda(), full[:, :2 * C], a=a)
    assert (full[:, 2 * C:] == 7).all()
    return to_np(full[:, :2 * C]), None if a is None else to_np(a)


def check_backward(dgu, a, da, ck, cs, dtype):
    C = da.shape[1]
    g, u = o.kept(ck, cs)
    ea, eg, eu = o.swiglu_bounds(da, g, u, HALF[dtype])
    dg, du = o.swiglu_bwd(da, g, u)
    for got, ref, e in ((dgu[:, :C], dg, eg), (dgu[:, C:], du, eu), (a, o.swiglu(g, u), ea)):
        if got is not None:
            bad = ~(np.abs(got - ref) <= e)
            assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R, C", SHAPES)
def test_backward(q, R, C, dtype):  # noqa: F811
    ck, cs = o.keep((rng(25, R, C).standard_normal((R, 2 * C)) * 4).astype(np.float32))
    dd, df = tensor(rng(26, R, C).standard_normal((R, C)) * 1e-3, dtype)
    for again, pad in ((True, 0), (False, 3)):
        dgu, a = backward(q, dd, ck, cs, again, pad)
        check_backward(dgu, a, df, ck, cs, dtype)


def test_backward_extremes(q):  # noqa: F811
    C = 256
    gu = np.concatenate([np.linspace(-200, 200, 2 * C).reshape(2, C), rng(27).standard_normal((2, C))], axis=1)
    ck, cs = o.keep(gu.astype(np.float32))
    dd, df = tensor(rng(28).standard_normal((2, C)), F32)
    dgu, a = backward(q, dd, ck, cs, True)
    check_backward(dgu, a, df, ck, cs, F32)


def test_backward_of_what_was_not_finite(q):  # noqa: F811
    C = 256
    ck, cs = o.keep(rng(29).standard_normal((2, 2 * C)).astype(np.float32))
    cs[0, 1], ck[0, 128:256] = np.nan, 0
    dd, _ = tensor(np.ones((2, C)), F32)
    dgu, _ = backward(q, dd, ck, cs, False)
    assert np.isnan(dgu[0, 128:256]).all() and np.isnan(dgu[0, C + 128:]).all()
    assert np.isfinite(dgu[0, :128]).all() and np.isfinite(dgu[1]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_views(q, dtype):  # noqa: F811
    """Inputs with odd strides and offsets; rows beside them are not read."""
    C = 333
    full = np.full((9, 2 * C + 5), np.nan, np.float32)
    full[2:7, 3:3 + 2 * C] = rng(30).standard_normal((5, 2 * C))
    gd, gf = tensor(full, dtype)
    gd, gf = gd[2:7, 3:3 + 2 * C], np.ascontiguousarray(gf[2:7, 3:3 + 2 * C])
    check_forward(make(q, gd, C, a=1, ck=1, cs=1), gf, dtype)
    check_forward(make(q, gd, C, aq=1, sa=1), gf, dtype)
    ck, cs = o.keep(gf)
    full = np.full((9, C + 5), np.nan, np.float32)
    full[2:7, 3:3 + C] = rng(31).standard_normal((5, C))
    dd, df = tensor(full, dtype)
    dgu, a = backward(q, dd[2:7, 3:3 + C], ck, cs, True, pad=1)
    check_backward(dgu, a, np.ascontiguousarray(df[2:7, 3:3 + C]), ck, cs, dtype)


def test_gradient_against_differences(q):  # noqa: F811
    """dgu from the calls against differences of the forward pass around the
    kept values: sum(da a) moves by dgu times a small step."""
    R, C, h = 4, 200, 2.0 ** -7
    ck, cs = o.keep((rng(32).standard_normal((R, 2 * C)) * 2).astype(np.float32))
    g, u = o.kept(ck, cs)
    gu = torch.from_numpy(np.concatenate([g, u], axis=1)).cuda()
    dd, df = tensor(rng(33).standard_normal((R, C)), F32)
    dgu, a = backward(q, dd, ck, cs, True)

    def forward(x):
        out = torch.empty((R, C), device="cuda")
        q.qsg_swiglu_int8_store_fwd(x, a=out)
        return to_np(out).astype(np.float64)

    assert np.allclose(a, forward(gu), rtol=1e-6, atol=1e-7)
    for half in range(2):
        step = torch.zeros_like(gu)
        step[:, half * C:(half + 1) * C] = h
        slope = (forward(gu + step) - forward(gu - step)) / (2 * h) * df
        # a second difference of silu is at most 0.5, a third at most 0.31: h^2 / 6 of it, and the forward pass's
        # roundings (2^-22 of the values) over the step
        tol = np.abs(df) * (h * h / 6 * 0.35 * (np.abs(u) + 1) + (np.abs(o.swiglu(g, u)) + np.abs(u) + 1) * 2.0 ** -20 / h)
        assert (np.abs(dgu[:, half * C:(half + 1) * C] - slope) <= tol).all()


def test_empty(q):  # noqa: F811
    for R, C in ((0, 5), (3, 0)):
        gu = torch.empty((R, 2 * C), dtype=BF, device="cuda")
        got = make(q, gu, C, a=1, aq=1, sa=1, ck=1, cs=1)
        assert (got["sa"] == 1).all()
        q.qsg_swiglu_int8_store_bwd(torch.empty((R, C), dtype=BF, device="cuda"),
                                    torch.empty((R, 2 * C), dtype=torch.int8, device="cuda"),
                                    torch.empty((R, 2 * -(-C // 128)), device="cuda"), gu)


def test_past_32_bits(q):  # noqa: F811
    """Offsets past 2^32 bytes and 2^31 elements in a matrix of many rows."""
    R, C = 530_000, 4096
    gu = torch.zeros((R, 2 * C), dtype=BF, device="cuda")
    at = [0, 262_143, 262_144, R - 1]
    for i, r in enumerate(at):
        gu[r] = torch.linspace(-3, 3 + i, 2 * C, device="cuda").to(BF)
    ck = torch.empty((R, 2 * C), dtype=torch.int8, device="cuda")
    cs = torch.empty((R, 2 * C // 128), device="cuda")
    a = torch.empty((R, C), dtype=BF, device="cuda")
    q.qsg_swiglu_int8_store_fwd(gu, a=a, ck=ck, cs=cs)
    for r in at:
        got = {"a": to_np(a[r:r + 1]), "ck": to_np(ck[r:r + 1]), "cs": to_np(cs[r:r + 1])}
        check_forward(got, gu[r:r + 1].float().cpu().numpy(), BF)
    assert int((cs != 1).sum()) == len(at) * 2 * C // 128
    da = a
    da.fill_(0.5)
    gu.fill_(9.0)
    q.qsg_swiglu_int8_store_bwd(da, ck, cs, gu)
    for r in at:
        check_backward(to_np(gu[r:r + 1]), None, np.full((1, C), 0.5), to_np(ck[r:r + 1]), to_np(cs[r:r + 1]), BF)
    assert int((gu != 0).any(dim=1).sum()) == len(at)


@pytest.mark.parametrize("R, C", [(3, 1111), (300, 512), (2, 33001)])
def test_fp32_far_gates(q, R, C):  # noqa: F811
    """fp32 keeps its bits however far the gate is from 0, where a rounded
    exponent would cost |g| of them."""
    x = rng(34, R, C).standard_normal((R, 2 * C))
    x[:, :C] = rng(35, R, C).uniform(-100, 100, (R, C))
    gd, gf = tensor(x, F32)
    g, u = gf[:, :C], gf[:, C:]
    bound = o.swiglu_bounds(None, g, u, HALF[F32], o.sigmoid_error_f32)[0]
    for outs in (dict(a=1), dict(a=1, aq=1, sa=1, ck=1, cs=1)):
        bad = ~(np.abs(make(q, gd, C, **outs)["a"] - o.swiglu(g, u)) <= bound)
        assert not bad.any(), (int(bad.sum()), g[bad][:4])
    ck, cs = o.keep(gf)
    g, u = o.kept(ck, cs)
    dd, df = tensor(rng(36, R, C).standard_normal((R, C)), F32)
    dgu, a = backward(q, dd, ck, cs, True)
    bounds = o.swiglu_bounds(df, g, u, HALF[F32], o.sigmoid_error_f32)
    for got, ref, e in zip((a, dgu[:, :C], dgu[:, C:]), (o.swiglu(g, u), *o.swiglu_bwd(df, g, u)), bounds):
        bad = ~(np.abs(got - ref) <= e)
        assert not bad.any(), (int(bad.sum()), g[bad][:4])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R, C", [(257, 2049), (300, 4104), (257, 8192), (260, 8193), (257, 14337), (258, 16384)])
def test_copy_of_many_rows(q, R, C, dtype):  # noqa: F811
    """More than 256 rows of 2049 columns and more hold a row's INT8 copy in
    fewer threads than few rows do."""
    gd, gf = tensor(rng(37, R, C).standard_normal((R, 2 * C)) * 4, dtype)
    check_forward(make(q, gd, C, a=1, aq=1, sa=1, ck=1, cs=1), gf, dtype)
    check_forward(make(q, gd, C, aq=1, sa=1), gf, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gates_at_the_ends(q, dtype):  # noqa: F811
    """Infinities, NaN and the largest finite gates, as g / (1 + exp(-g)) has them."""
    top = torch.finfo(dtype).max
    g = np.array([np.inf, -np.inf, np.nan, top, -top, 1e30, -1e30, 128, -128, 0.0, 2.0 ** -126])
    want = np.array([np.inf, np.nan, np.nan, top / 2, 0, 5e29, 0, 64, 0, 0, 2.0 ** -128])
    gd, gf = tensor(np.concatenate([g, np.full(11, 0.5)])[None], dtype)
    want[5] = gf[0, 5] / 2
    a = make(q, gd, 11, a=1, aq=1, sa=1)["a"][0]
    assert np.array_equal(a, make(q, gd, 11, a=1)["a"][0], equal_nan=True)
    assert np.array_equal(a, want, equal_nan=True)
