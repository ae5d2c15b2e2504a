"""What the INT8 calls refuse, on the CPU: the C entry points' own checks (no
call here reaches a launch), and the binding's."""

import pytest
import torch

import quantize_scaled_gemm_amd as q
from helpers import build_library, lib_is_stale
from test_binding_cpu import BF, F32, U8, raises
from test_binding_cpu import Dev as Stand

I8 = torch.int8


@pytest.fixture(scope="module")
def lib():
    if lib_is_stale():
        build_library()
    return q.load_library()


# plausible addresses: never dereferenced, every call below is refused
QUANT = dict(x=4096, dtype=1, rows=64, cols=96, ld=96, q=8192, s=64, qt=12288, st=128, ws=256)
GEMM = dict(a=4096, sa=64, b=8192, sb=128, M=64, N=96, K=256, lda=256, ldb=256, bias=512, bdt=1, c=12288, cdt=1, ldc=96)
WGRAD = dict(dy=4096, T=64, N=96, lddy=96, q=8192, s=64, K=128, ldq=128, c=12288, cdt=0, ldc=128, acc=0)
FWD = dict(gu=4096, dtype=1, rows=4, cols=200, ld=400, a=8192, aq=12288, sa=64, ck=16384, cs=128)
BWD = dict(da=4096, dtype=1, rows=4, cols=200, ldda=200, ck=8192, cs=64, dgu=12288, lddgu=400, a=16384)
BIG = 1 << 30


@pytest.mark.parametrize("base, kw, status", [
    (QUANT, dict(dtype=2), -1), (QUANT, dict(x=None), -1), (QUANT, dict(rows=-1), -1), (QUANT, dict(ld=95), -1),
    (QUANT, dict(x=4097), -3), (QUANT, dict(q=None, s=None, qt=None, st=None), -1), (QUANT, dict(s=None), -1),
    (QUANT, dict(q=None), -1), (QUANT, dict(st=None), -1), (QUANT, dict(qt=None), -1), (QUANT, dict(s=66), -3),
    (QUANT, dict(st=66), -3), (QUANT, dict(ws=None), -1), (QUANT, dict(ws=258), -3), (QUANT, dict(rows=BIG), -4),
    (QUANT, dict(cols=BIG, ld=BIG), -4), (QUANT, dict(qt=8192), -1), (QUANT, dict(q=4096), -1), (QUANT, dict(st=64), -1),
    (GEMM, dict(cdt=3), -1), (GEMM, dict(bdt=3), -1), (GEMM, dict(K=-1), -1), (GEMM, dict(K=131072, lda=1 << 20, ldb=1 << 20), -4),
    (GEMM, dict(lda=255), -1), (GEMM, dict(ldb=255), -1), (GEMM, dict(ldc=95), -1), (GEMM, dict(a=None), -1),
    (GEMM, dict(b=None), -1), (GEMM, dict(sa=None), -1), (GEMM, dict(sb=None), -1), (GEMM, dict(c=None), -1),
    (GEMM, dict(sa=66), -3), (GEMM, dict(sb=66), -3), (GEMM, dict(c=12289), -3), (GEMM, dict(c=12290, cdt=0), -3),
    (GEMM, dict(bias=513), -3), (GEMM, dict(bias=514, bdt=0), -3), (GEMM, dict(M=(1 << 26) + 1), -4),
    (GEMM, dict(N=(1 << 26) + 1, ldc=1 << 27), -4), (GEMM, dict(M=1 << 26, N=1 << 26, ldc=1 << 26), -4),
    (GEMM, dict(c=4096), -1),
    (WGRAD, dict(cdt=2), -1), (WGRAD, dict(T=-1), -1), (WGRAD, dict(cdt=1, acc=1), -4), (WGRAD, dict(c=None), -1),
    (WGRAD, dict(ldc=127), -1), (WGRAD, dict(c=12290), -3), (WGRAD, dict(dy=None), -1), (WGRAD, dict(q=None), -1),
    (WGRAD, dict(s=None), -1), (WGRAD, dict(lddy=95), -1), (WGRAD, dict(ldq=127), -1), (WGRAD, dict(dy=4097), -3),
    (WGRAD, dict(s=66), -3), (WGRAD, dict(N=1 << 25, lddy=1 << 25), -4), (WGRAD, dict(K=(1 << 26) + 1, ldq=1 << 27), -4),
    (FWD, dict(dtype=2), -1), (FWD, dict(gu=None), -1), (FWD, dict(cols=-1), -1), (FWD, dict(ld=399), -1),
    (FWD, dict(gu=4097), -3), (FWD, dict(a=None, aq=None, sa=None, ck=None, cs=None), -1), (FWD, dict(sa=None), -1),
    (FWD, dict(aq=None), -1), (FWD, dict(cs=None), -1), (FWD, dict(ck=None), -1), (FWD, dict(a=8193), -3),
    (FWD, dict(sa=66), -3), (FWD, dict(cs=130), -3), (FWD, dict(a=4096), -1), (FWD, dict(ck=12288), -1),
    (FWD, dict(aq=8192), -1), (FWD, dict(sa=128), -1), (FWD, dict(cols=BIG, ld=2 * BIG), -4), (FWD, dict(rows=BIG), -4),
    (BWD, dict(dtype=2), -1), (BWD, dict(da=None), -1), (BWD, dict(ldda=199), -1), (BWD, dict(lddgu=399), -1),
    (BWD, dict(ck=None), -1), (BWD, dict(cs=None), -1), (BWD, dict(dgu=None), -1), (BWD, dict(cs=66), -3),
    (BWD, dict(dgu=12289), -3), (BWD, dict(a=16385), -3), (BWD, dict(dgu=4096), -1), (BWD, dict(a=4096), -1),
    (BWD, dict(a=12288), -1), (BWD, dict(rows=BIG), -4), (BWD, dict(cols=BIG, ldda=BIG, lddgu=2 * BIG), -4),
])
def test_library_refuses(lib, base, kw, status):
    call = {id(QUANT): lib.qsg_quantize_int8, id(GEMM): lib.qsg_gemm_int8, id(WGRAD): lib.qsg_wgrad_int8,
            id(FWD): lib.qsg_swiglu_int8_store_fwd, id(BWD): lib.qsg_swiglu_int8_store_bwd}[id(base)]
    assert set(kw) <= set(base)
    assert call(*dict(base, **kw).values(), None) == status
    assert lib.qsg_last_error()


def test_nothing_to_do_is_no_error(lib):
    assert lib.qsg_gemm_int8(*dict(GEMM, M=0).values(), None) == 0
    assert lib.qsg_wgrad_int8(*dict(WGRAD, N=0).values(), None) == 0
    assert lib.qsg_swiglu_int8_store_fwd(*dict(FWD, rows=0, sa=None).values(), None) == 0
    assert lib.qsg_swiglu_int8_store_bwd(*dict(BWD, cols=0).values(), None) == 0


@pytest.mark.parametrize("kw", [
    dict(cols=0, s=None), dict(cols=0, s=None, ws=None), dict(cols=0, s=None, qt=None, st=None),
    dict(rows=0, st=None), dict(rows=0, st=None, q=None, s=None)])
def test_empty_codes_without_the_scales_that_are_there(lib, kw):
    """Of a matrix without columns every row has a scale, which is written; of
    one without rows every column of the transposed copy."""
    assert lib.qsg_quantize_int8(*dict(QUANT, **kw).values(), None) == -1
    assert b"go together" in lib.qsg_last_error()


def test_workspace_sizes(lib):
    for bad in ((-1, 4), (4, -1), (BIG, 4), (4, BIG)):
        with pytest.raises(q.QsgError):
            q.qsg_quantize_int8_workspace(*bad)
    assert q.qsg_quantize_int8_workspace(0, 9) == q.qsg_quantize_int8_workspace(9, 0) == 0
    sizes = [q.qsg_quantize_int8_workspace(r, 100) for r in (1, 2, 511, 512, 513, 5000, BIG - 1)]
    assert sizes == sorted(sizes) and sizes[0] >= 400
    assert q.qsg_quantize_int8_workspace(300, 101) >= q.qsg_quantize_int8_workspace(300, 100)


class Dev(Stand):
    """A stand-in that may have an address (no call here reaches a launch)."""

    def __init__(self, shape, dtype, strides=None, cuda=True, device=0):
        super().__init__(shape, dtype, strides, cuda)
        self.device_index = device

    def data_ptr(self):
        return 4096

    def element_size(self):
        return {BF: 2, F32: 4, U8: 1, I8: 1}[self.dtype]

    def get_device(self):
        return self.device_index


def test_binding_refuses():
    x, c8, f = Dev((6, 300), BF), Dev((6, 300), I8), lambda n: Dev((n,), F32)
    quant = q.qsg_quantize_int8
    raises(lambda: quant(Dev((6, 300), torch.float16), q=c8, s=f(6)), "unsupported input dtype")
    raises(lambda: quant(x, q=Dev((6, 300), U8), s=f(6)), "q must be i8")
    raises(lambda: quant(x, q=Dev((6, 299), I8), s=f(6)), "q must hold exactly 1800")
    raises(lambda: quant(x, q=c8, s=f(5)), "s must hold exactly 6")
    raises(lambda: quant(x, q=c8), "s is required")
    raises(lambda: quant(x, s=f(6)), "q is required")
    raises(lambda: quant(x, qt=c8, st=f(300)), "workspace is required")
    raises(lambda: quant(x, qt=c8, st=f(300), workspace=Dev((7199,), U8)), "workspace must hold at least 7200")
    raises(lambda: quant(Dev((6, 300), BF, strides=(200, 1)), q=c8, s=f(6)), "the rows overlap")
    raises(lambda: quant(Dev((6, 300), BF, strides=(1, 6)), q=c8, s=f(6)), "last dimension must be contiguous")
    raises(lambda: quant(x, q=Dev((6, 300), I8, strides=(301, 1)), s=f(6)), "q must be contiguous")
    gemm, a, b, c = q.qsg_gemm_int8, Dev((4, 64), I8), Dev((9, 64), I8), Dev((4, 9), BF)
    raises(lambda: gemm(Dev((4, 64), U8), f(4), b, f(9), c), "A must hold INT8 codes")
    raises(lambda: gemm(a, f(4), Dev((9, 64), BF), f(9), c), "B must hold INT8 codes")
    raises(lambda: gemm(a, f(4), Dev((9, 65), I8), f(9), c), "K mismatch")
    raises(lambda: gemm(a, f(4), b, f(9), Dev((9, 4), BF)), "C is 9x4")
    raises(lambda: gemm(a, f(4), b, f(9), Dev((4, 9), torch.float16)), "unsupported")
    raises(lambda: gemm(a, f(3), b, f(9), c), "sa must hold exactly 4")
    raises(lambda: gemm(a, f(4), b, f(8), c), "sb must hold exactly 9")
    raises(lambda: gemm(a, f(4), b, f(9), c, bias=f(4)), "bias must hold exactly 9")
    raises(lambda: gemm(a, f(4), b, f(9), Dev((4, 9), BF, strides=(5, 1))), "C: the rows overlap")
    wgrad, dy, qq = q.qsg_wgrad_int8, Dev((7, 16), BF), Dev((7, 32), I8)
    raises(lambda: wgrad(Dev((7, 16), F32), qq, f(7), Dev((16, 32), F32)), "bf16 dY")
    raises(lambda: wgrad(dy, Dev((7, 32), U8), f(7), Dev((16, 32), F32)), "q must hold INT8 codes")
    raises(lambda: wgrad(dy, Dev((6, 32), I8), f(6), Dev((16, 32), F32)), "token count mismatch")
    raises(lambda: wgrad(dy, qq, f(7), Dev((32, 16), F32)), "C is 32x16")
    raises(lambda: wgrad(dy, qq, f(32), Dev((16, 32), F32)), "s must hold exactly 7")
    fwd, gu = q.qsg_swiglu_int8_store_fwd, Dev((5, 400), BF)
    raises(lambda: fwd(Dev((5, 401), BF), a=Dev((5, 200), BF)), "gu has 401 columns")
    raises(lambda: fwd(gu, a=Dev((5, 200), F32)), "a must be bf16")
    raises(lambda: fwd(gu, aq=Dev((5, 200), I8)), "sa is required")
    raises(lambda: fwd(gu, ck=Dev((5, 200), I8), cs=f(20)), "ck must hold exactly 2000")
    raises(lambda: fwd(gu, ck=Dev((5, 400), I8), cs=f(10)), "cs must hold exactly 20")
    bwd, da, ck = q.qsg_swiglu_int8_store_bwd, Dev((5, 200), BF), Dev((5, 400), I8)
    raises(lambda: bwd(da, ck, f(20), None), "dgu is required")
    raises(lambda: bwd(da, ck, f(20), Dev((5, 200), BF)), "dgu is 5x200")
    raises(lambda: bwd(da, ck, f(20), Dev((5, 400), F32)), "dgu must be")
    raises(lambda: bwd(da, ck, f(19), Dev((5, 400), BF)), "cs must hold exactly 20")
    raises(lambda: bwd(da, None, f(20), Dev((5, 400), BF)), "ck is required")
    raises(lambda: bwd(da, ck, f(20), Dev((5, 400), BF), a=Dev((5, 200), F32)), "a must be bf16")


def test_binding_refuses_other_devices(monkeypatch):
    """The library launches on the current device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f = Dev((4,), F32)
    there = dict(device=1)
    calls = [
        lambda: q.qsg_quantize_int8(Dev((4, 8), BF, **there), q=Dev((4, 8), I8, **there), s=Dev((4,), F32, **there)),
        lambda: q.qsg_quantize_int8(Dev((4, 8), BF), q=Dev((4, 8), I8), s=Dev((4,), F32, **there)),
        lambda: q.qsg_gemm_int8(Dev((4, 8), I8), f, Dev((4, 8), I8, **there), f, Dev((4, 4), BF)),
        lambda: q.qsg_wgrad_int8(Dev((4, 8), BF), Dev((4, 8), I8), f, Dev((8, 8), F32, **there)),
        lambda: q.qsg_swiglu_int8_store_fwd(Dev((4, 8), BF), a=Dev((4, 4), BF, **there)),
        lambda: q.qsg_swiglu_int8_store_bwd(Dev((4, 4), BF, **there), Dev((4, 8), I8), Dev((4, 2), F32), Dev((4, 8), BF)),
    ]
    for call in calls:
        raises(call, "on device 1, the current device is 0|is on device 1, the call's first tensor on device 0|"
               "is on device 0, the call's first tensor on device 1")
