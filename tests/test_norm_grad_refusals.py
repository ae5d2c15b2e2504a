"""What the norm and clipping calls refuse, on the CPU: the C entry points'
own checks (no call here reaches a launch), and the binding's."""

import ctypes

import pytest
import torch

import quantize_scaled_gemm_amd as q
from helpers import build_library, lib_is_stale
from test_binding_cpu import BF, F32, U8, raises
from test_binding_cpu import Dev as Stand

NAN, INF = float("nan"), float("inf")
F64 = torch.float64


@pytest.fixture(scope="module")
def lib():
    if lib_is_stale():
        build_library()
    return q.load_library()


# plausible addresses: never dereferenced, every call below is refused
A = dict(x=4096, residual=8192, dtype=1, rows=128, cols=256, ldx=256, ldr=256, gamma=64, gdtype=1, eps=1e-5,
         recipe=(q.MXFP8, q.E4M3, 0, q.MX_CEIL), scale=None, h=12288, ldh=256, rstd=16384, y=None, q=32, s=64, qt=32,
         st=64, amax=None)


def fwd(lib, **kw):
    a = dict(A, **kw)
    rec = None if a["recipe"] is None else ctypes.byref(q.Recipe(*a["recipe"]))
    return lib.qsg_rmsnorm_quantize(a["x"], a["residual"], a["dtype"], a["rows"], a["cols"], a["ldx"], a["ldr"],
                                    a["gamma"], a["gdtype"], a["eps"], rec, a["scale"], a["h"], a["ldh"], a["rstd"],
                                    a["y"], a["q"], a["s"], a["qt"], a["st"], a["amax"], None)


TW, DL, B1 = (q.TENSORWISE, q.E4M3, 0, 0), (q.DELAYED, q.E4M3, 0, 0), (q.BLOCK_1X128, q.E4M3, 0, 0)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=2), -1), (dict(gdtype=5), -1), (dict(x=None), -1), (dict(gamma=None), -1), (dict(rows=-1), -1),
    (dict(ldx=255), -1), (dict(ldr=255), -1), (dict(ldh=255), -1), (dict(eps=-1e-9), -1), (dict(eps=NAN), -1),
    (dict(eps=INF), -1), (dict(x=4097), -3), (dict(residual=8193), -3), (dict(h=12289), -3), (dict(rstd=16386), -3),
    (dict(gamma=65), -3), (dict(gamma=66, gdtype=0), -3), (dict(h=None), -1),
    (dict(h=8192, ldr=512), -1), (dict(h=4096, ldx=512), -1),              # in place needs one leading dimension
    (dict(q=None, qt=None), -1), (dict(rstd=None), -1),                    # qt needs rstd
    (dict(recipe=None), -1), (dict(recipe=None, q=None, qt=None), -1),     # FP8 without a recipe; no output
    (dict(recipe=(q.BLOCK_128X128, 0, 0, 0)), -4), (dict(recipe=(9, 0, 0, 0)), -1), (dict(recipe=(-1, 0, 0, 0)), -1),
    (dict(recipe=(q.MXFP8, 2, 0, 0)), -1), (dict(recipe=(q.MXFP8, 0, 65, 0)), -1),
    (dict(recipe=(q.MXFP8, 0, 0, 2)), -1), (dict(s=None), -1), (dict(st=None), -1),
    (dict(cols=240, ldx=256), -2), (dict(rows=48), -2), (dict(recipe=B1, rows=96), -2),
    (dict(recipe=B1, cols=192), -2), (dict(recipe=B1, s=66), -3),
    (dict(recipe=TW, s=None), -1), (dict(recipe=TW, s=66), -3), (dict(recipe=TW, qt=None, rstd=None), -1),
    (dict(recipe=TW, amax=64), -1), (dict(amax=64), -1), (dict(recipe=DL), -1), (dict(recipe=DL, scale=66), -3),
    (dict(cols=(1 << 24) + 32, ldx=1 << 25, ldr=1 << 25, ldh=1 << 25), -4),
    (dict(recipe=DL, scale=64, amax=66), -3), (dict(y=33, recipe=DL, scale=64), -3),
])
def test_forward_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status, (kw, lib.qsg_last_error())


def test_empty_calls_launch_nothing(lib):
    assert fwd(lib, rows=0, x=None, residual=None, gamma=None, h=None) == 0
    assert fwd(lib, cols=0, x=None, q=None, qt=None) == 0
    assert fwd(lib, recipe=None, rows=0, q=None, qt=None) == 0
    assert lib.qsg_rmsnorm_bwd(None, None, None, 1, 5, 0, 0, 0, 0, None, 1, None, None, 0, None, 0, None, None) == 0
    assert lib.qsg_rmsnorm_bwd(None, None, None, 1, 0, 5, 5, 5, 5, None, 1, None, None, 5, None, 0, None, None) == 0


B = dict(dy=4096, h=8192, dres=12288, dtype=1, rows=8, cols=256, lddy=256, ldh=256, lddres=256, gamma=64, gdtype=0,
         rstd=64, dx=16384, lddx=256, dgamma=128, acc=0, ws=256)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), -1), (dict(gdtype=-1), -1), (dict(dy=None), -1), (dict(h=None), -1), (dict(gamma=None), -1),
    (dict(rstd=None), -1), (dict(dx=None), -1), (dict(ws=None), -1), (dict(rows=-1), -1), (dict(cols=-2), -1),
    (dict(lddy=128), -1), (dict(ldh=128), -1), (dict(lddres=128), -1), (dict(lddx=128), -1), (dict(dy=4097), -3),
    (dict(h=8193), -3), (dict(dres=12289), -3), (dict(dx=16385), -3), (dict(gamma=66), -3), (dict(rstd=66), -3),
    (dict(dgamma=130), -3), (dict(ws=258), -3), (dict(dx=8192), -1),        # dx may not be h
    (dict(dx=4096, lddy=512), -1), (dict(dx=12288, lddres=512), -1),
    (dict(cols=(1 << 24) + 8, lddy=1 << 25, ldh=1 << 25, lddres=1 << 25, lddx=1 << 25), -4),
])
def test_backward_refuses(lib, kw, status):
    a = dict(B, **kw)
    assert lib.qsg_rmsnorm_bwd(a["dy"], a["h"], a["dres"], a["dtype"], a["rows"], a["cols"], a["lddy"], a["ldh"],
                               a["lddres"], a["gamma"], a["gdtype"], a["rstd"], a["dx"], a["lddx"], a["dgamma"],
                               a["acc"], a["ws"], None) == status, (kw, lib.qsg_last_error())


def test_backward_workspace(lib):
    assert lib.qsg_rmsnorm_bwd_workspace(-1, 4) == -1
    assert lib.qsg_rmsnorm_bwd_workspace(0, 4) == 0 == lib.qsg_rmsnorm_bwd_workspace(4, 0)
    # a row of dgamma at least for every row of a few
    assert lib.qsg_rmsnorm_bwd_workspace(1, 1000) >= 4000
    with pytest.raises(q.QsgError, match="negative"):
        q.qsg_rmsnorm_bwd_workspace(4, -1)


def plan(lib, entries, room=None):
    arr = (q.Grad * max(1, len(entries)))(*[q.Grad(*e, 0) for e in entries])
    n = ctypes.c_int64(0)
    rc = lib.qsg_grad_plan(arr, len(entries), None, ctypes.byref(n))
    if rc:
        return rc, None
    need = n.value
    chunks = (q.Grad * max(1, need))()
    n.value = need if room is None else room
    rc = lib.qsg_grad_plan(arr, len(entries), chunks, ctypes.byref(n))
    return rc, [(c.g, c.out, c.n, c.dtype) for c in chunks[:need]]


def test_plan_cuts_every_element_once(lib):
    entries = [(1 << 20, 1 << 30, 100001, q.F32), (1 << 40, None, 1, q.BF16), (None, None, 0, q.F32),
               ((1 << 41) + 2, (1 << 42) + 2, 70000, q.BF16)]
    rc, chunks = plan(lib, entries)
    assert rc == 0
    at = 0
    for g, out, n, dtype in entries:
        esz = 4 if dtype == q.F32 else 2
        left, off = n, 0
        while left:
            cg, co, cn, cd = chunks[at]
            assert cd == dtype and 0 < cn <= left
            assert cg == g + off * esz and co == (None if out is None else out + off * esz)
            left, off, at = left - cn, off + cn, at + 1
    assert at == len(chunks)


def test_plan_refuses(lib):
    for entry, status in (((64, 64, 4, 7), -1), ((64, 64, -1, 0), -1), ((None, 64, 4, 0), -1), ((66, 64, 4, 0), -3),
                          ((64, 66, 4, 0), -3), ((65, 64, 4, 1), -3)):
        assert plan(lib, [entry])[0] == status, entry
    assert plan(lib, [(64, 64, 100000, 0)], room=1)[0] == -1
    assert lib.qsg_grad_plan(None, 1, None, ctypes.byref(ctypes.c_int64(0))) == -1
    assert lib.qsg_grad_plan(None, 0, None, None) == -1
    assert plan(lib, []) == (0, [])


def test_clipping_refuses(lib):
    assert lib.qsg_grad_sumsq(None, 1, 64, 64, None) == -1
    assert lib.qsg_grad_sumsq(64, -1, 64, 64, None) == -1
    assert lib.qsg_grad_sumsq(64, 1, None, 64, None) == -1
    assert lib.qsg_grad_sumsq(64, 1, 64, None, None) == -1
    assert lib.qsg_grad_sumsq(64, 1, 68, 64, None) == -3
    assert lib.qsg_grad_clip(None, 1, 64, 1.0, None, None) == -1
    assert lib.qsg_grad_clip(64, 1, None, 1.0, None, None) == -1
    assert lib.qsg_grad_clip(64, 1, 64, -1.0, None, None) == -1
    assert lib.qsg_grad_clip(64, 1, 64, NAN, None, None) == -1
    assert lib.qsg_grad_clip(64, 1, 60, 1.0, None, None) == -3
    assert lib.qsg_grad_clip(64, 1, 64, 1.0, 66, None) == -3


class Dev(Stand):
    """A stand-in for a GPU tensor whose address may be asked for."""

    def data_ptr(self):
        return 4096


@pytest.fixture
def no_call(lib, monkeypatch):
    """A library whose calls that launch must not be reached."""

    class Lib:
        qsg_rmsnorm_bwd_workspace = lib.qsg_rmsnorm_bwd_workspace
        qsg_grad_plan = lib.qsg_grad_plan

        def __getattr__(self, name):
            def reached(*args):
                raise AssertionError(f"the binding must reject this call before it reaches {name}")

            return reached

    monkeypatch.setattr(q, "load_library", Lib)
    monkeypatch.setattr(q, "_stream", lambda stream: None)


def test_binding_checks_the_forward(no_call):
    x, g, r = Dev((64, 256), BF), Dev((256,), BF), Dev((64,), F32)
    qq, s = Dev((64, 256), U8), Dev((64, 8), U8)
    M = q.MXFP8
    raises(lambda: q.qsg_rmsnorm_quantize(x, Dev((255,), BF), 1e-5, M, q=qq, s=s), "gamma must hold exactly 256")
    raises(lambda: q.qsg_rmsnorm_quantize(x, Dev((256,), U8), 1e-5, M, q=qq, s=s), "unsupported input dtype")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, residual=Dev((64, 255), BF), q=qq, s=s), "residual is 64x255")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, residual=x, h=Dev((64, 256), F32), q=qq, s=s), "h must be")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, rstd=Dev((63,), F32), q=qq, s=s), "rstd must hold exactly 64")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, y=Dev((64, 256), F32)), "y must be bf16")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, q=Dev((64, 255), U8), s=s), "q must hold exactly")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, q=qq, s=Dev((64, 7), U8)), "s must hold exactly 512")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, M, qt=qq, st=Dev((256, 1), U8)), "st must hold exactly 512")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, q.TENSORWISE, q=qq, s=Dev((2,), F32), rstd=r), "s must hold exactly 3")
    raises(lambda: q.qsg_rmsnorm_quantize(x, g, 1e-5, q.DELAYED, q=qq), "scale is required")
    raises(lambda: q.qsg_rmsnorm_quantize(Dev((64, 256), BF, strides=(0, 1)), g, 1e-5, M, q=qq, s=s), "rows overlap")
    raises(lambda: q.qsg_rmsnorm_quantize(Dev((64, 256), BF, strides=(1, 64)), g, 1e-5, M, q=qq, s=s), "contiguous")


def test_binding_checks_the_backward(no_call):
    x, g, r = Dev((64, 256), BF), Dev((256,), BF), Dev((64,), F32)
    ws = Dev((q.qsg_rmsnorm_bwd_workspace(64, 256),), U8)
    ws.element_size = lambda: 1
    raises(lambda: q.qsg_rmsnorm_bwd(x, Dev((64, 128), BF), g, r, x, workspace=ws), "h is 64x128")
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, r, Dev((64, 256), F32), workspace=ws), "dx must be")
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, Dev((64,), BF), x, workspace=ws), "rstd must be f32")
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, r, x, dres=Dev((1, 256), BF), workspace=ws), "dres is 1x256")
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, r, x, dgamma=Dev((256,), BF), workspace=ws), "dgamma must be f32")
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, r, x), "workspace is required")
    small = Dev((16,), U8)
    small.element_size = lambda: 1
    raises(lambda: q.qsg_rmsnorm_bwd(x, x, g, r, x, workspace=small), "workspace must hold at least")


def test_binding_checks_the_gradients(no_call):
    a = Dev((4, 4), F32)
    a.device = "cuda:0"
    b = Dev((4, 4), BF)
    b.device = "cuda:0"
    raises(lambda: q.qsg_grad_plan([a], [a, a]), "1 gradients, but 2 outputs")
    raises(lambda: q.qsg_grad_plan([Dev((4,), F32, cuda=False)]), "gradient 0 must live on the GPU")
    c = Dev((4, 4), F32, strides=(8, 1))
    c.device = "cuda:0"
    raises(lambda: q.qsg_grad_plan([a, c]), "gradient 1 must be contiguous")
    raises(lambda: q.qsg_grad_plan([a], [b]), "output 0 must have the shape and type")

    p = q.GradPlan(Dev((32,), U8), 1, [], [])
    ws = Dev((q.GRAD_WORKSPACE_BYTES,), U8)
    ws.element_size = lambda: 1
    raises(lambda: q.qsg_grad_sumsq(p, Dev((1,), F32), ws), "sumsq must be f64")
    raises(lambda: q.qsg_grad_clip(p, Dev((1,), F64), 1.0, Dev((1,), F64)), "norm_out must be f32")
