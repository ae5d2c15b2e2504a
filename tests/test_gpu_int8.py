"""INT8 on the GPU: copies bit-exact against the oracle, products within the
roundings of their scaling, the weight gradient within those of its sum."""

import numpy as np
import pytest
import torch

from helpers import to_np
from oracle import int8 as o

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def rng(*k):
    return np.random.Generator(np.random.PCG64([43, *k]))


def tensor(x, dtype):
    """(GPU tensor of the type, its values as binary32)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)
    return t.cuda(), t.float().numpy()


def same(got, want):
    return np.array_equal(np.ascontiguousarray(got).view(np.uint8), np.ascontiguousarray(want).view(np.uint8))


def same_scales(got, want):
    return np.array_equal(got, want, equal_nan=True)


def quantize(q, x, rows=True, cols=True, **kw):
    R, C = x.shape
    out = {}
    if rows:
        out["q"] = torch.full((R, C), 99, dtype=torch.int8, device="cuda")
        out["s"] = torch.full((R,), -7.0, device="cuda")
    if cols:
        out["qt"] = torch.full((C, R), 99, dtype=torch.int8, device="cuda")
        out["st"] = torch.full((C,), -7.0, device="cuda")
        kw["workspace"] = torch.full((q.qsg_quantize_int8_workspace(R, C),), 255, dtype=torch.uint8, device="cuda")
    q.qsg_quantize_int8(x, **out, **kw)
    return {k: to_np(v) for k, v in out.items()}


def check_copies(got, x, name=""):
    if "q" in got:
        rq, rs = o.quantize(x)
        assert same_scales(got["s"], rs), name
        assert same(got["q"], rq), name
    if "qt" in got:
        rq, rs = o.quantize(np.ascontiguousarray(x.T))
        assert same_scales(got["st"], rs), name
        assert same(got["qt"], rq), name


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 15), (129, 16), (64, 127), (17, 129), (300, 256), (33, 257), (2, 512), (70, 513),
          (9, 1000), (31, 1024), (5, 1025), (130, 2048), (3, 2049), (6, 4096), (4, 4097), (3, 8192), (2, 8193),
          (2, 16384), (1, 16385), (2, 32768), (2, 32769), (3, 40003), (1000, 63), (513, 65), (2051, 40), (255, 2056),
          (257, 4095), (700, 2500), (520, 5001), (300, 9000), (3000, 600), (2101, 1500), (8300, 2060), (1, 2100), (2, 9001)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_copies(q, shape, dtype):
    x = rng(1, *shape).standard_normal(shape) * 10.0 ** rng(2, *shape).integers(-4, 4, (shape[0], 1))
    xd, xf = tensor(x, dtype)
    check_copies(quantize(q, xd), xf)


@pytest.mark.parametrize("rows, cols", [(True, False), (False, True)])
def test_one_copy(q, rows, cols):
    xd, xf = tensor(rng(3).standard_normal((200, 333)), BF)
    check_copies(quantize(q, xd, rows, cols), xf)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_views(q, dtype):
    """Odd strides and offsets; what lies beside the view is not read."""
    full = rng(4).standard_normal((67, 411)).astype(np.float32)
    view = full[3:60, 5:304].copy()
    full[:] = np.nan
    full[3:60, 5:304] = view
    xd, _ = tensor(full, dtype)
    xf = torch.from_numpy(view).to(dtype).float().numpy()
    check_copies(quantize(q, xd[3:60, 5:304]), xf)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 700, 3000, 40000])
def test_special_values(q, cols, dtype):
    """Rows and columns of zeros, of the smallest and largest values, with an
    infinity or a NaN, and ties."""
    x = rng(5, cols).standard_normal((16, cols)).astype(np.float32)
    x[1] = 0
    x[2] = -0.0
    x[3, 5] = np.inf
    x[4, 6] = -np.inf
    x[5, cols - 1] = np.nan
    x[6] *= np.float32(1e-38)
    x[7] = np.where(np.arange(cols) % 2, 1e-40, -3e-41)
    x[8, 0], x[8, 1] = 3.3e38, -3.3e38
    x[9] = np.round(x[9] * 20) + 0.5
    x[9, 0] = 127
    x[:, 9] = 0
    x[3:6, 9] = 0
    xd, xf = tensor(x, dtype)
    check_copies(quantize(q, xd), xf)


def test_nan_payloads(q):
    """A NaN's low bits do not reach the codes."""
    bits = np.full((2, 300), 0x3F800000, np.uint32)
    bits[0, 10], bits[1, 299] = 0x7F8000FF, 0xFFC0AB5D
    x = torch.from_numpy(bits.view(np.float32)).cuda()
    got = quantize(q, x)
    assert np.isnan(got["s"]).all() and not got["q"].any()
    assert np.isnan(got["st"][[10, 299]]).all() and not got["qt"][[10, 299]].any()


def test_many_columns(q):
    """More columns than one launch has threads for their scales."""
    cols = 2 ** 28 + 70
    x = torch.zeros((1, cols), dtype=BF, device="cuda")
    at = torch.tensor([0, 63, 64, 2 ** 27 - 1, 2 ** 27, 2 ** 28 - 1, 2 ** 28, 2 ** 28 + 69], device="cuda")
    v = torch.tensor([1, -2, 3, -4, 5, -6, 7, -8], device="cuda").to(BF)
    x[0, at] = v
    qt, st = torch.full((cols, 1), 9, dtype=torch.int8, device="cuda"), torch.full((cols,), -1.0, device="cuda")
    ws = torch.empty(q.qsg_quantize_int8_workspace(1, cols), dtype=torch.uint8, device="cuda")
    q.qsg_quantize_int8(x, qt=qt, st=st, workspace=ws)
    assert torch.equal(qt[at, 0], 127 * torch.sign(v.float()).to(torch.int8))
    assert torch.equal(st[at], v.float().abs() / 127)
    qt[at], st[at] = 0, 1.0
    assert not qt.any() and (st == 1).all()


def test_empty(q):
    for shape in ((0, 5), (5, 0), (0, 0)):
        got = quantize(q, torch.empty(shape, dtype=BF, device="cuda"))
        assert (got["s"] == 1).all() and (got["st"] == 1).all()


def test_empty_with_addresses(q):
    """A caller of the C interface may pass the addresses of copies that hold
    nothing."""
    buf = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    st = torch.zeros(64, device="cuda")
    p = buf.data_ptr()
    q.qsg_quantize_int8(torch.empty((0, 64), dtype=BF, device="cuda"), q=p, s=p + 1024, qt=p + 2048, st=st,
                        workspace=p + 3328)
    s = torch.zeros(64, device="cuda")
    q.qsg_quantize_int8(torch.empty((64, 0), dtype=BF, device="cuda"), q=p, s=s, qt=p + 2048, st=p + 1024,
                        workspace=p + 3328)
    assert (st == 1).all() and (s == 1).all() and not buf.any()


def test_workspace_serves_smaller_shapes(q):
    ws = torch.empty(q.qsg_quantize_int8_workspace(700, 300), dtype=torch.uint8, device="cuda")
    for R, C in ((700, 300), (699, 300), (511, 299), (3, 300), (1, 1)):
        assert q.qsg_quantize_int8_workspace(R, C) <= ws.numel()
        xd, xf = tensor(rng(6, R).standard_normal((R, C)), F32)
        qt = torch.empty((C, R), dtype=torch.int8, device="cuda")
        st = torch.empty(C, device="cuda")
        q.qsg_quantize_int8(xd, qt=qt, st=st, workspace=ws)
        check_copies({"qt": to_np(qt), "st": to_np(st)}, xf)


def test_more_rows_than_a_launch(q):
    """Row indices and element offsets past 32 bits: 2^31 + elements."""
    R, C = (1 << 21) * 16 + 5, 72
    x = torch.zeros((R, C), dtype=BF, device="cuda")
    at = [0, 1 << 21, (1 << 21) * 16 - 1, (1 << 21) * 16, R - 1]
    for i, r in enumerate(at):
        x[r] = torch.arange(C, device="cuda").to(BF) - i
    got = {"q": torch.empty((R, C), dtype=torch.int8, device="cuda"), "s": torch.empty(R, device="cuda")}
    q.qsg_quantize_int8(x, **got)
    for r in at:
        rq, rs = o.quantize(x[r:r + 1].float().cpu().numpy())
        assert same(to_np(got["q"][r:r + 1]), rq) and same_scales(to_np(got["s"][r:r + 1]), rs), r
    assert int((got["s"] != 1).sum()) == len(at)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def codes(k, *shape):
    return rng(7, k, *shape).integers(-128, 128, shape).astype(np.int8)


def product(q, M, N, K, out, bias=None, pad=0, extreme=False):
    a, b = codes(1, M, K), codes(2, N, K)
    if extreme:
        a[:], b[:] = -128, -128
    sa, sb = rng(8, M).random(M).astype(np.float32), rng(9, N).random(N).astype(np.float32) * 0.01
    ad = torch.full((M, K + pad), 77, dtype=torch.int8, device="cuda")[:, pad:]
    bd = torch.full((N, K + pad), 77, dtype=torch.int8, device="cuda")[:, pad:]
    ad.copy_(torch.from_numpy(a))
    bd.copy_(torch.from_numpy(b))
    cfull = torch.full((M, N + pad), 5.0, dtype=out, device="cuda")
    c = cfull[:, pad:]
    bias_d, bias_f = (None, None) if bias is None else tensor(rng(10, N).standard_normal(N) * 100, bias)
    q.qsg_gemm_int8(ad, torch.from_numpy(sa).cuda(), bd, torch.from_numpy(sb).cuda(), c, bias=bias_d)
    got, ref = to_np(c).astype(np.float64), o.gemm(a, sa, b, sb, bias_f)
    bad = np.abs(got - ref) > o.gemm_bound(ref, bias_f, HALF[out])
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    assert (cfull[:, :pad] == 5.0).all()


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [
    (1, 1, 1), (1, 16, 64), (1, 300, 4096), (2, 17, 127), (7, 64, 128), (15, 33, 129), (16, 128, 1000), (17, 40, 256),
    (31, 100, 2049), (32, 64, 512), (33, 50, 640), (61, 130, 1536), (64, 256, 4100), (65, 128, 64), (100, 5, 300),
    (128, 128, 128), (129, 257, 255), (200, 300, 1111), (1021, 96, 384), (5, 1000, 14336), (300, 1000, 2048)])
def test_product(q, M, N, K, out):
    product(q, M, N, K, out)


@pytest.mark.parametrize("bias", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [(1, 129, 256), (40, 64, 384), (130, 201, 512)])
def test_product_bias(q, M, N, K, bias):
    product(q, M, N, K, BF, bias)
    product(q, M, N, K, F32, bias)


@pytest.mark.parametrize("out, bias", [(BF, None), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("M, N, K, pad", [
    (1, 12300, 1040, 0), (4, 12288, 512, 16), (5, 12300, 640, 0), (16, 12301, 2064, 0),      # few rows, many columns
    (3, 4100, 2064, 0), (16, 900, 4112, 16), (17, 900, 4112, 0), (32, 4100, 656, 0),         # few rows and columns
    (20, 12300, 528, 0), (32, 12289, 400, 32), (33, 4100, 1040, 0), (64, 900, 16, 0),        # up to 64 rows
    (61, 10250, 1040, 0), (64, 12289, 256, 16), (100, 4100, 2064, 0), (128, 4096, 1024, 0),
    (61, 28700, 4096, 0), (16, 12301, 4096, 0), (40, 4100, 4096, 0), (7, 900, 8192, 0), (16, 130, 12288, 0),  # far rows
    (33, 10300, 4000, 96), (20, 900, 4064, 32),                                              # in a wider matrix
    (300, 1000, 144, 0), (450, 4100, 784, 0), (511, 4097, 400, 16), (1021, 3100, 528, 0), (900, 4100, 112, 0),
    (3, 800, 333, 0), (40, 700, 333, 0), (16, 7000, 129, 0), (200, 700, 333, 0), (53, 608, 1227, 5), (1000, 3201, 333, 3), (900, 4100, 100, 1)])  # any alignment
def test_product_forms(q, M, N, K, pad, out, bias):
    """Every way that the sizes choose, with ragged edges and short K."""
    test_large_product(q, M, N, K, pad, out, bias)


@pytest.mark.parametrize("out, bias", [(BF, None), (F32, None), (BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("M, N, K, pad", [
    (4096, 2048, 512, 0), (2900, 4098, 256, 0), (4250, 4096, 768, 16),  # 128 tiles of 256 x 256, ragged, a tail launch
    (8500, 4100, 1280, 32), (2900, 4097, 512, 0), (4000, 2304, 640, 0), (3000, 4096, 512, 8)])
def test_large_product(q, M, N, K, pad, out, bias):
    """Every output against exact sums, which a product in 64 bits gives."""
    g = torch.Generator("cuda").manual_seed(M + N + K)
    a = torch.randint(-128, 128, (M, K + pad), device="cuda", dtype=torch.int8, generator=g)[:, :K]
    b = torch.randint(-128, 128, (N, K + pad), device="cuda", dtype=torch.int8, generator=g)[:, :K]
    sa, sb = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    bd = None if bias is None else (torch.randn(N, device="cuda", generator=g) * 1000).to(bias)
    full = torch.full((M, N + 3), 7.0, device="cuda", dtype=out)
    q.qsg_gemm_int8(a, sa, b, sb, full[:, :N], bias=bd)
    c = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    p = c.abs()
    if bd is not None:
        c += bd.double()
        p += bd.double().abs()
    e = 2.0 ** -24 * (4 * p + c.abs())
    assert ((full[:, :N].double() - c).abs() <= e + HALF[out] * (c.abs() + e)).all()
    assert (full[:, N:] == 7).all()
    dense = torch.empty((M, N), device="cuda", dtype=out)
    q.qsg_gemm_int8(a, sa, b, sb, dense, bias=bd)
    assert torch.equal(dense, full[:, :N])


@pytest.mark.parametrize("pad", [1, 3, 16])
@pytest.mark.parametrize("M, N, K", [(3, 50, 300), (50, 40, 256), (150, 140, 333)])
def test_product_views(q, M, N, K, pad):
    product(q, M, N, K, BF, pad=pad)
    product(q, M, N, K, F32, pad=pad)


@pytest.mark.parametrize("M", [1, 40, 130])
def test_largest_sum(q, M):
    """K = 131071 codes of -128: the largest sum, just below 2^31."""
    product(q, M, 20, 131071, F32, extreme=True)


@pytest.mark.parametrize("M", [1, 70])
def test_product_without_k(q, M):
    c = torch.full((M, 9), 5.0, device="cuda")
    bias = torch.arange(9.0, device="cuda")
    e = torch.empty((M, 0), dtype=torch.int8, device="cuda")
    f = torch.empty((9, 0), dtype=torch.int8, device="cuda")
    q.qsg_gemm_int8(e, torch.ones(M, device="cuda"), f, torch.ones(9, device="cuda"), c, bias=bias)
    assert (c == bias).all()


@pytest.mark.parametrize("M", [2, 80])
def test_nan_scales_reach_their_rows(q, M):
    a, b = torch.zeros((M, 256), dtype=torch.int8, device="cuda"), torch.zeros((40, 256), dtype=torch.int8, device="cuda")
    sa, sb = torch.ones(M, device="cuda"), torch.ones(40, device="cuda")
    sa[1] = float("nan")
    sb[39] = float("nan")
    c = torch.empty((M, 40), dtype=BF, device="cuda")
    q.qsg_gemm_int8(a, sa, b, sb, c)
    nan = torch.isnan(c)
    want = torch.zeros_like(nan)
    want[1], want[:, 39] = True, True
    assert (nan == want).all() and (c[~want] == 0).all()


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------
def wgrad(q, T, N, K, out, accumulate=False, whole=False, pad=0):
    qq = codes(3, T, K)
    s = rng(11, T).random(T).astype(np.float32) * 0.1
    dy = rng(12, T, N).standard_normal((T, N)) * 1e-3
    if whole:  # whole numbers of few bits: every sum is exact
        qq = rng(13, T, K).integers(-8, 9, (T, K)).astype(np.int8)
        s = 2.0 ** rng(14, T).integers(0, 3, T).astype(np.float32)
        dy = rng(15, T, N).integers(-4, 5, (T, N))
    dyd, dyf = tensor(np.pad(dy, ((0, 0), (pad, 0))), BF)
    dyf = dyf[:, pad:]
    qd = torch.full((T, K + pad), 77, dtype=torch.int8, device="cuda")[:, pad:]
    qd.copy_(torch.from_numpy(qq))
    c0 = rng(16).standard_normal((N, K)).astype(np.float32) if accumulate else np.full((N, K), 5, np.float32)
    if whole:
        c0 = np.round(c0)
    c = torch.from_numpy(c0).to(out).cuda()
    q.qsg_wgrad_int8(dyd[:, pad:], qd, torch.from_numpy(s).cuda(), c, accumulate=accumulate)
    ref, bound = o.wgrad(dyf, qq, s)
    if accumulate:
        ref = ref + c0
        bound = bound + 2.0 ** -24 * np.abs(ref)
    got = to_np(c).astype(np.float64)
    if whole:
        bound = np.zeros_like(ref)
        if out == BF:
            ref = torch.from_numpy(ref).float().to(BF).double().numpy()
    else:
        bound = bound + HALF[out] * (np.abs(ref) + bound)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


WGRAD = [(1, 1, 1), (1, 8, 16), (7, 33, 40), (16, 256, 256), (47, 8, 16), (48, 64, 128), (49, 264, 272), (63, 100, 257),
         (64, 256, 300), (65, 512, 16), (97, 24, 48), (144, 300, 256), (145, 256, 512), (200, 130, 77), (777, 264, 400),
         (1000, 40, 304), (1500, 72, 333), (2600, 72, 333), (2113, 520, 500), (1601, 600, 650), (1601, 1100, 1050), (600, 2050, 2100)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T, N, K", WGRAD)
def test_wgrad(q, T, N, K, out):
    wgrad(q, T, N, K, out)
    wgrad(q, T, N, K, out, whole=True)


@pytest.mark.parametrize("T, N, K", [(130, 72, 96), (333, 257, 300), (512, 256, 256)])
def test_wgrad_accumulates(q, T, N, K):
    wgrad(q, T, N, K, F32, accumulate=True)
    wgrad(q, T, N, K, F32, accumulate=True, whole=True)


@pytest.mark.parametrize("pad", [1, 8, 16])
def test_wgrad_views(q, pad):
    wgrad(q, 150, 136, 160, F32, whole=True, pad=pad)
    wgrad(q, 150, 130, 140, BF, whole=True, pad=pad)


def test_wgrad_without_tokens(q):
    dy, qq = torch.empty((0, 3), dtype=BF, device="cuda"), torch.empty((0, 5), dtype=torch.int8, device="cuda")
    s = torch.empty(0, device="cuda")
    c = torch.full((3, 5), 2.0, device="cuda")
    q.qsg_wgrad_int8(dy, qq, s, c, accumulate=True)
    assert (c == 2).all()
    q.qsg_wgrad_int8(dy, qq, s, c)
    assert (c == 0).all()


def test_wgrad_nan_scale(q):
    """A token that could not be quantized makes the whole gradient NaN, its
    codes of 0 notwithstanding."""
    for K in (32, 33):
        dy = torch.ones((70, 24), dtype=BF, device="cuda")
        qq = torch.ones((70, K), dtype=torch.int8, device="cuda")
        s = torch.ones(70, device="cuda")
        qq[69], s[69] = 0, float("nan")
        c = torch.zeros((24, K), device="cuda")
        q.qsg_wgrad_int8(dy, qq, s, c)
        assert torch.isnan(c).all()


@pytest.mark.parametrize("N, K", [(2048, 4096), (2001, 2050), (500, 2100), (24, 33)])
def test_wgrad_largest_values(q, N, K):
    """A token whose maximum is bf16's largest value: 128 times its scale is
    not finite, its codes times its scale are.  One product a sum, so exact."""
    top = torch.finfo(BF).max
    T, g = 70, torch.Generator(device="cuda").manual_seed(5)
    s = torch.ones(T, device="cuda")
    s[69] = float(np.float32(top) / np.float32(127))
    qq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda", generator=g)
    qq[69, 0], qq[69, 1], qq[69, 2] = 127, -127, 0
    dy = torch.zeros((T, N), dtype=BF, device="cuda")
    dy[69] = 2.0 ** torch.randint(-6, -2, (N,), device="cuda", generator=g)
    x = (qq[69].float() * s[69]).to(BF).float()
    assert torch.isfinite(x).all() and x[0] == top
    c = torch.full((N, K), 5.0, device="cuda")
    q.qsg_wgrad_int8(dy, qq, s, c)
    assert torch.equal(c, dy[69].float()[:, None] * x[None, :])


# ---------------------------------------------------------------------------
# offsets beyond 32 bits
# ---------------------------------------------------------------------------
def far_rows(rows):
    return torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")


def test_copies_beyond_32_bits(q):
    rows, cols = 263000, 16400  # 4.3e9 values
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    at = far_rows(rows)
    v = torch.from_numpy(rng(31).standard_normal((5, cols))).to(BF).cuda()
    x[at] = v
    qq, s = torch.empty((rows, cols), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    qt, st = torch.empty((cols, rows), dtype=torch.int8, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(q.qsg_quantize_int8_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    q.qsg_quantize_int8(x, q=qq, s=s, qt=qt, st=st, workspace=ws)
    vf = to_np(v)
    check_copies({"q": to_np(qq[at]), "s": to_np(s[at])}, vf)
    check_copies({"qt": to_np(qt[:, at].contiguous()), "st": to_np(st)}, vf)
    assert int(torch.count_nonzero(s == 1)) == rows - 5
    for part in qt.chunk(64):  # the other rows are zeros
        part[:, at] = 0
        assert not part.any()


def test_activation_beyond_32_bits(q):
    rows, cols = 132000, 16400  # 4.3e9 values of gu
    gu = torch.zeros((rows, 2 * cols), dtype=BF, device="cuda")
    at = far_rows(rows)
    gu[at] = torch.from_numpy(rng(32).standard_normal((5, 2 * cols))).to(BF).cuda()
    nb = -(-cols // 128)

    def run(gu):
        n = gu.shape[0]
        o = [torch.empty((n, cols), dtype=BF, device="cuda"), torch.empty((n, cols), dtype=torch.int8, device="cuda"),
             torch.empty(n, device="cuda"), torch.empty((n, 2 * cols), dtype=torch.int8, device="cuda"),
             torch.empty((n, 2 * nb), device="cuda")]
        q.qsg_swiglu_int8_store_fwd(gu, a=o[0], ck=o[3], cs=o[4])
        q.qsg_swiglu_int8_store_fwd(gu, aq=o[1], sa=o[2])
        dgu, a = torch.empty_like(gu), torch.empty_like(o[0])
        q.qsg_swiglu_int8_store_bwd(o[0], o[3], o[4], dgu, a)
        return [*o, dgu, a]

    for big, small in zip(run(gu), run(gu[at].contiguous())):
        assert torch.equal(big[at], small)


@pytest.mark.parametrize("N, K", [(64, 16400), (61, 16401)])
def test_products_beyond_32_bits(q, N, K):
    rows = 263000  # 4.3e9 codes
    a = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    at = far_rows(rows)
    ca = codes(33, 5, K)
    a[at] = torch.from_numpy(ca).cuda()
    cb = codes(34, N, K)
    one, c = torch.ones(rows, device="cuda"), torch.full((rows, N), 5.0, device="cuda")
    q.qsg_gemm_int8(a, one, torch.from_numpy(cb).cuda(), one[:N], c)
    want = (ca.astype(np.int64) @ cb.astype(np.int64).T).astype(np.float32)
    assert same(to_np(c[at]), want)
    c[at] = 0
    assert not c.any()
    # the weight gradient of powers of two: every sum is exact
    dy = torch.zeros((rows, N), dtype=BF, device="cuda")
    dy[at] = 2.0 ** torch.arange(5, device="cuda", dtype=torch.float32).to(BF)[:, None]
    w = torch.empty((N, K), device="cuda")
    q.qsg_wgrad_int8(dy, a, one, w)
    assert same(to_np(w), np.broadcast_to((ca * 2.0 ** np.arange(5)[:, None]).sum(0), (N, K)).astype(np.float32))


@pytest.mark.parametrize("out, accumulate", [(BF, False), (F32, False), (F32, True)])
@pytest.mark.parametrize("T, N, K, pad", [
    (1, 2056, 4112, 0), (47, 2056, 4112, 16), (49, 2304, 3856, 0), (96, 2048, 4096, 0), (144, 2056, 4112, 8),
    (145, 4096, 2320, 16), (337, 2056, 4112, 0),                                   # direct loads, 128 tiles and more
    (200, 2000, 2500, 0), (333, 2001, 2050, 3), (70, 1100, 1050, 5), (333, 600, 650, 1), (600, 130, 333, 0),
    (2600, 40, 70, 7), (5000, 33, 129, 1)])                                        # other tiles
def test_wgrad_into_views(q, T, N, K, pad, out, accumulate):
    """C with rows further apart: every output, exactly (whole numbers of few
    bits), and nothing beside it written."""
    g = torch.Generator("cuda").manual_seed(T + N + K)
    dy = torch.randint(-4, 5, (T, N + pad), device="cuda", generator=g).to(BF)[:, :N]
    qq = torch.randint(-8, 9, (T, K + pad), device="cuda", dtype=torch.int8, generator=g)[:, :K]
    s = 2.0 ** torch.randint(0, 3, (T,), device="cuda", generator=g).float()
    full = torch.randint(-9, 10, (N, K + pad), device="cuda", generator=g).to(out)
    before = full.clone()
    q.qsg_wgrad_int8(dy, qq, s, full[:, :K], accumulate=accumulate)
    want = dy.double().t().contiguous() @ (qq.double() * s.double()[:, None])
    if accumulate:
        want += before[:, :K].double()
    assert torch.equal(full[:, :K], want.to(out))
    assert torch.equal(full[:, K:], before[:, K:])
