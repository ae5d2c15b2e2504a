"""qsg_rmsnorm_quantize and qsg_rmsnorm_bwd against the 64-bit oracle.

Forward: h is bit-exact (one addition, one rounding); rstd is within the error
of a binary32 sum of squares; every output after it is bit-exact, because y is
two binary32 products of h, the rstd that the call returns and gamma, and the
FP8 copies of y are those of the quantizer oracle.  Backward: element by
element within oracle.norm.norm_bwd_bound."""

import numpy as np
import pytest

import oracle
from helpers import to_dev, to_np

pytestmark = pytest.mark.gpu

EPS = 1e-5
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def torch_type(dtype):
    import torch

    return torch.bfloat16 if dtype == "bf16" else torch.float32


def make(rng, rows, cols, dtype, std=1.0, ld=None, offset=0):
    """A rows x cols view with leading dimension ld, `offset` elements into its
    buffer; the elements around it are NaN."""
    import torch

    ld = ld or cols
    buf = torch.full((offset + max(rows, 1) * ld + 8,), float("nan"), dtype=torch_type(dtype), device="cuda")
    t = buf[offset:offset + max(rows, 1) * ld].view(max(rows, 1), ld)[:rows, :cols]
    v = (rng.standard_normal((rows, cols)) * std).astype(np.float32)
    if cols > 4:
        v[:, rng.integers(0, cols, max(1, cols // 100))] *= 20
    t.copy_(to_dev(v))
    return t


def longest(cols):
    """Additions in a row that one binary32 partial sum may see: a lane's chunks
    (64 lanes for at most 16 chunks each, else 256), a tail, and the tree."""
    return 8 * max(min(16, -(-cols // 512)), -(-cols // 2048)) + 16


def weights(rng, cols, dtype):
    return make(rng, 1, cols, dtype, 0.1).view(-1) + 1


def quantizers(recipe, y, fmt, margin, rule, scale):
    """(q, s, qt, st, amax) of the oracle for y."""
    rows, cols = y.shape
    if recipe == "mx":
        d = oracle.mx_quantize(y, fmt, rule, margin, rowwise=cols % 32 == 0, colwise=rows % 32 == 0)
        return d.get("q"), d.get("s"), d.get("qt"), d.get("st"), None
    if recipe == "1x128":
        d = oracle.block_quantize_1x128(y, fmt, margin, rowwise=cols % 128 == 0, colwise=rows % 128 == 0)
        return d.get("q"), d.get("s"), d.get("qt"), d.get("st"), None
    if recipe == "tensorwise":
        a, b, am, sc, si = oracle.quantize_tensorwise(y, fmt, margin)
        return a, np.array([am, sc, si], np.float32), b, None, None
    a, b = oracle.cast_transpose(y, scale, fmt)
    return a, None, b, None, oracle.amax(y)


def same(got, want, what):
    got, want = to_np(got), np.asarray(want)
    if got.dtype.kind == "f":
        got, want = np.ascontiguousarray(got, np.float32).view(np.uint32), np.ascontiguousarray(want, np.float32).view(np.uint32)
    assert got.shape == want.shape or got.size == want.size, what
    bad = np.flatnonzero(got.ravel() != want.ravel())
    assert bad.size == 0, f"{what}: {bad.size} of {got.size} differ, first at {bad[:4]}"


def forward(q, rng, rows, cols, dtype, recipe, fmt="e4m3", residual=True, t=True, y=False, gamma="bf16", margin=0,
            rule="ceil", ld=None, offset=0, inplace=None, x=None, r=None, w=None, eps=EPS, check=True):
    """One call, checked against the oracle; returns its outputs."""
    import torch

    codes = {"mx": q.MXFP8, "1x128": q.BLOCK_1X128, "delayed": q.DELAYED, "tensorwise": q.TENSORWISE, None: None}
    x = make(rng, rows, cols, dtype, 1.0, ld, offset) if x is None else x
    if residual and r is None:
        r = make(rng, rows, cols, dtype, 2.0, ld, offset)
    w = weights(rng, cols, gamma) if w is None else w
    x0, r0 = to_np(x).copy(), to_np(r).copy() if residual else None
    h = {"x": x, "r": r}.get(inplace)
    if h is None and residual:
        h = torch.empty_like(x)
    u8 = dict(dtype=torch.uint8, device="cuda")
    o = dict(rstd=torch.empty(rows, device="cuda"), h=h)
    if y:
        o["y"] = torch.empty((rows, cols), dtype=x.dtype, device="cuda")
    scale = None
    if recipe:
        # copies land in guarded buffers: one byte off either end is seen
        guard = torch.full((2, rows * cols + 2), 0xA5, **u8)
        o["q"] = guard[0, 1:-1].view(rows, cols)
        if t:
            o["qt"] = guard[1, 1:-1].view(cols, rows)
        if recipe == "mx":
            o["s"] = torch.empty((rows, cols // 32), **u8)
            o["st"] = torch.empty((cols, rows // 32), **u8) if t else None
        elif recipe == "1x128":
            o["s"] = torch.empty((rows, cols // 128), device="cuda")
            o["st"] = torch.empty((cols, rows // 128), device="cuda") if t else None
        elif recipe == "tensorwise":
            o["s"] = torch.empty(3, device="cuda")
        else:
            scale = torch.full((1,), 40.0, device="cuda")
            o["amax_out"] = torch.full((1,), -1.0, device="cuda")
    q.qsg_rmsnorm_quantize(x, w, eps, codes[recipe], q.FMT[fmt], residual=r if residual else None, scale=scale,
                           margin=margin, mx_rule=q.MX_CEIL if rule == "ceil" else q.MX_OCP_FLOOR, **o)
    torch.cuda.synchronize()
    if not check:
        return o
    hv = x0
    if residual:
        hv = to_np(torch.from_numpy(x0 + r0).to(x.dtype))
        same(o["h"], hv, "h")
    if inplace != "x":
        same(x, x0, "x is read only")
    if residual and inplace != "r":
        same(r, r0, "the residual is read only")
    rstd = to_np(o["rstd"]).astype(np.float64)
    want = oracle.norm.rstd(hv, eps)
    tol = (longest(cols) / 2 + 5) * U
    assert (np.abs(rstd - want) <= tol * want).all(), np.abs(rstd / want - 1).max()
    y32 = oracle.norm.normed_f32(hv, to_np(o["rstd"]), to_np(w))
    if y:
        same(o["y"], to_np(torch.from_numpy(y32).to(x.dtype)), "y")
    if recipe:
        wq, ws, wqt, wst, wamax = quantizers(recipe, y32, fmt, margin, rule, np.float32(40.0))
        same(o["q"], wq, "q")
        if ws is not None:
            same(o["s"], ws, "s")
        if t:
            same(o["qt"], wqt, "qt")
            if wst is not None:
                same(o["st"], wst, "st")
        if wamax is not None:
            same(o["amax_out"], np.float32([wamax]), "amax")
        g = guard.cpu().numpy()
        assert (g[:, 0] == 0xA5).all() and (g[:, -1] == 0xA5).all(), "a byte outside q or qt was written"
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("recipe, rows, cols, t", [
    ("mx", 1, 32, False), ("mx", 1, 4096, False), ("mx", 3, 96, False), ("mx", 32, 32, True), ("mx", 96, 160, True),
    ("mx", 160, 1056, True), ("mx", 256, 512, True), ("mx", 5, 7168, False), ("mx", 2, 16416, False),
    ("1x128", 1, 128, False), ("1x128", 2, 7168, False), ("1x128", 128, 128, True), ("1x128", 256, 384, True),
    ("1x128", 3, 16512, False), ("1x128", 128, 1152, True),
    ("delayed", 1, 1, True), ("delayed", 2, 7, True), ("delayed", 65, 131, True), ("delayed", 128, 256, True),
    ("delayed", 129, 1111, False), ("delayed", 300, 2049, True), ("delayed", 4, 16391, True),
    ("delayed", 3, 20011, False),
    ("tensorwise", 1, 5, True), ("tensorwise", 1, 4096, False), ("tensorwise", 200, 300, True),
    ("tensorwise", 67, 4100, False), ("tensorwise", 2, 16400, True),
    (None, 1, 1, False), (None, 33, 515, False), (None, 2, 40003, False),
])
def test_forward(q, dtype, recipe, rows, cols, t):
    forward(q, np.random.default_rng([rows, cols]), rows, cols, dtype, recipe, t=t, y=recipe is None)


@pytest.mark.parametrize("dtype, rows, cols", [
    ("bf16", 1500, 520), ("bf16", 1100, 1040), ("bf16", 1030, 2056), ("bf16", 1027, 4104), ("bf16", 2100, 264),
    ("bf16", 1025, 8199), ("bf16", 2100, 1040), ("bf16", 2051, 4103), ("f32", 2049, 1111), ("f32", 1030, 2056), ("f32", 1100, 520), ("bf16", 100, 520), ("bf16", 100, 2056),
    ("bf16", 40, 4104), ("bf16", 30, 8200), ("f32", 30, 4104), ("f32", 20, 8200)])
def test_forward_row_variants(q, dtype, rows, cols):
    """Every way that a row is held: a wave or a workgroup, 1 to 16 chunks a
    lane, with a tail of single elements where cols % 8 is not 0."""
    forward(q, np.random.default_rng(cols), rows, cols, dtype, "delayed", t=False, y=True)


@pytest.mark.parametrize("recipe, fmt, margin, rule", [
    ("mx", "e5m2", 0, "ceil"), ("mx", "e4m3", 2, "ceil"), ("mx", "e4m3", 0, "ocp"), ("mx", "e5m2", 1, "ocp"),
    ("1x128", "e5m2", 3, "ceil"), ("tensorwise", "e5m2", 1, "ceil"), ("delayed", "e5m2", 0, "ceil")])
def test_forward_recipe_knobs(q, recipe, fmt, margin, rule):
    for dtype, t in (("bf16", True), ("f32", False)):
        forward(q, np.random.default_rng(5), 128, 256, dtype, recipe, fmt=fmt, margin=margin, rule=rule, t=t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("recipe, rows, cols, t", [("mx", 64, 96, True), ("1x128", 128, 256, True),
                                                   ("delayed", 37, 83, True), ("tensorwise", 19, 1000, False)])
def test_forward_views(q, dtype, recipe, rows, cols, t):
    """Rows further apart than cols, bases off by one element, fp32 weights on
    bf16 data and the reverse, with and without a residual."""
    rng = np.random.default_rng(7)
    for residual in (False, True):
        for ld, offset in ((cols + 3, 1), (cols + 8, 0), (cols, 3)):
            forward(q, rng, rows, cols, dtype, recipe, t=t, y=True, ld=ld, offset=offset, residual=residual,
                    gamma="f32" if dtype == "bf16" else "bf16")


@pytest.mark.parametrize("inplace", ["x", "r"])
@pytest.mark.parametrize("rows, cols, t", [(5, 256, False), (128, 1024, True), (2, 16512, False)])
def test_forward_in_place(q, inplace, rows, cols, t):
    forward(q, np.random.default_rng(9), rows, cols, "bf16", "mx", t=t, ld=cols + 8, inplace=inplace)


@pytest.mark.parametrize("recipe", ["mx", "1x128", "delayed", "tensorwise"])
@pytest.mark.parametrize("t", [False, True])
def test_forward_special_rows(q, recipe, t):
    """A row of zeros, tiny and large rows, one NaN, an infinity: the others
    are what they are without them (per-row and block scales), and the bad
    rows follow the formula."""
    rng = np.random.default_rng(11)
    x = make(rng, 128, 256, "f32")
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    o = forward(q, rng, 128, 256, "f32", recipe, x=x, residual=False, t=t)
    assert np.isfinite(to_np(o["rstd"])).all()
    x[5, 17] = float("nan")
    x[9, 200] = float("inf")
    o = forward(q, rng, 128, 256, "f32", recipe, x=x, residual=False, t=t, check=False)
    r = to_np(o["rstd"])
    assert np.isnan(r[5]) and r[9] == 0 and np.isfinite(np.delete(r, 5)).all()
    qq = to_np(o["q"])
    assert ((qq[5] & 0x7F) == 0x7F).all()
    assert (qq[9, 200] & 0x7F) == 0x7F and ((np.delete(qq[9], 200) & 0x7F) == 0).all()
    if recipe in ("mx", "1x128"):
        assert ((np.delete(qq, [5, 9], axis=0) & 0x7F) != 0x7F).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("recipe, fmt, margin, rule", [("mx", "e4m3", 0, "ceil"), ("mx", "e5m2", 0, "ceil"),
                                                       ("mx", "e4m3", 40, "ceil"), ("mx", "e4m3", 0, "ocp"),
                                                       ("1x128", "e4m3", 0, "ceil"), ("tensorwise", "e4m3", 0, "ceil")])
def test_forward_extreme_weights_and_rows(q, dtype, recipe, fmt, margin, rule):
    """Weights from the smallest subnormal to near the largest number, zeros
    among them, on rows from 1e-15 to 1e15: blocks whose values are subnormal,
    overflow to infinity, or are scaled by the outermost powers of two."""
    rng = np.random.default_rng(13)
    rows, cols = 256, 256
    x = make(rng, rows, cols, dtype)
    x *= to_dev((10.0 ** rng.integers(-15, 16, (rows, 1))).astype(np.float32)).to(x.dtype)
    x[64:96] = 0
    w = np.float32(2.0) ** rng.integers(-149, 127, cols).astype(np.float32) * rng.choice([-1, 1], cols)
    w[:64] = np.float32(2.0) ** rng.integers(-70, 70, 64).astype(np.float32)
    w[64:128] *= np.float32(2.0) ** rng.integers(-60, 0, 64).astype(np.float32)
    w[5], w[70], w[130] = 0.0, -0.0, 0.0
    w = to_dev(w.astype(np.float32))
    for t in (False, True):
        forward(q, rng, rows, cols, dtype, recipe, fmt=fmt, margin=margin, rule=rule, x=x, w=w, residual=False, t=t,
                eps=1e-30)


def test_forward_weights_that_are_not_finite(q):
    """An infinite and a NaN weight spoil their own columns and the blocks that
    hold them, and nothing else."""
    rng = np.random.default_rng(17)
    w = weights(rng, 256, "f32")
    w[40], w[200] = float("inf"), float("nan")
    for recipe in ("mx", "1x128"):
        o = forward(q, rng, 128, 256, "f32", recipe, w=w, check=False)
        qt = to_np(o["qt"])
        assert ((qt[200] & 0x7F) == 0x7F).all()
        assert ((qt[40] & 0x7F) == 0x7E).all()
        assert ((np.delete(qt, [40, 200], axis=0) & 0x7F) != 0x7F).all()


def test_forward_zero_row_without_eps_is_nan(q):
    import torch

    x = torch.zeros((2, 64), device="cuda")
    x[1] = 1
    y, rstd = torch.empty_like(x), torch.empty(2, device="cuda")
    q.qsg_rmsnorm_quantize(x, torch.ones(64, device="cuda"), 0.0, rstd=rstd, y=y)
    assert torch.isnan(y[0]).all() and (y[1] == 1).all() and rstd[1] == 1


def test_forward_empty(q):
    import torch

    for shape in ((0, 64), (4, 0)):
        x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        w = torch.ones(shape[1], device="cuda")
        qq = torch.empty(shape, device="cuda", dtype=torch.uint8)
        s = torch.full((3,), -1.0, device="cuda")
        q.qsg_rmsnorm_quantize(x, w, EPS, q.TENSORWISE, q=qq, s=s, rstd=torch.empty(shape[0], device="cuda"))
        assert s.tolist() == [0.0, 1.0, 1.0]
        am = torch.full((1,), -1.0, device="cuda")
        q.qsg_rmsnorm_quantize(x, w, EPS, q.DELAYED, q=qq, scale=torch.ones(1, device="cuda"), amax_out=am)
        assert am.item() == 0.0


def test_forward_offsets_past_32_bits(q):
    """Rows whose byte and element offsets pass 2^32 (a 4.3 GB stride)."""
    import torch

    ld, cols = (1 << 32) // 2 + 64, 256
    buf = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, cols), (ld, 1))
    rng = np.random.default_rng(3)
    x.copy_(to_dev(rng.standard_normal((3, cols)).astype(np.float32)))
    forward(q, rng, 3, cols, "bf16", "mx", x=x, residual=False, t=False)
    w = torch.ones(cols, device="cuda")
    dy = torch.as_strided(buf, (3, cols), (ld, 1))
    rstd = torch.ones(3, device="cuda")
    dx = torch.empty((3, cols), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(3, cols), dtype=torch.uint8, device="cuda")
    q.qsg_rmsnorm_bwd(dy, dy, w, rstd, dx, workspace=ws)
    close_dx(dx, to_np(x), to_np(x), np.ones(3), np.ones(cols), None, "bf16")


def test_more_than_2_32_elements(q):
    """Dense outputs past 2^32 bytes and elements: the last rows of a large call
    are those of a call on them alone."""
    import torch

    rows, cols, tail = (1 << 21) + 128, 2080, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 18):
        part.normal_(generator=g)
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")

    def call(x):
        r = x.shape[0]
        u8 = dict(dtype=torch.uint8, device="cuda")
        o = dict(rstd=torch.empty(r, device="cuda"), q=torch.empty((r, cols), **u8), s=torch.empty((r, cols // 32), **u8),
                 qt=torch.empty((cols, r), **u8), st=torch.empty((cols, r // 32), **u8))
        q.qsg_rmsnorm_quantize(x, w, EPS, q.MXFP8, **o)
        return o

    big, small = call(x), call(x[-tail:])
    for name in ("rstd", "q", "s"):
        assert torch.equal(big[name][-tail:], small[name]), name
    assert torch.equal(big["qt"][:, -tail:], small["qt"]) and torch.equal(big["st"][:, -tail // 32:], small["st"])
    # the byte transpose, and the backward pass in place of dy
    scale = torch.full((1,), 30.0, device="cuda")
    q.qsg_rmsnorm_quantize(x, w, EPS, q.DELAYED, rstd=big["rstd"], q=big["q"], qt=big["qt"], scale=scale)
    assert torch.equal(big["q"][-tail:].t(), big["qt"][:, -tail:])
    h, dy = x[-tail:].clone(), x[-tail:].clone()
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    q.qsg_rmsnorm_bwd(dy, h, w, small["rstd"], dy, workspace=ws)
    out = torch.empty_like(x)
    q.qsg_rmsnorm_bwd(x, x, w, big["rstd"], out, workspace=ws)
    assert torch.equal(out[-tail:], dy)


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def close_dx(dx, dy, h, rstd, w, dres, dtype):
    ref, _ = oracle.norm.norm_bwd(dy, h, rstd, w, dres)
    bound = oracle.norm.norm_bwd_bound(dy, h, rstd, w, dres, longest(np.shape(h)[1]), HALF[dtype])
    off = np.abs(to_np(dx).astype(np.float64) - ref)
    assert (off <= bound).all(), f"dx: {(off / np.maximum(bound, 1e-300)).max():.3g} times its bound"


def close_dgamma(dgamma, dy, h, rstd, start=None):
    """Partial sums over at most ceil(rows / groups) rows, then over groups / 32
    and 32: at most rows / 1024 + 70 additions in a chain (fewer rows than
    groups: none before the second)."""
    dy, n = np.asarray(dy, np.float64), np.asarray(h, np.float64) * np.asarray(rstd, np.float64)[:, None]
    ref, mag = (dy * n).sum(axis=0), np.abs(dy * n).sum(axis=0)
    if start is not None:
        ref, mag = ref + start, mag + np.abs(start)
    off = np.abs(to_np(dgamma).astype(np.float64) - ref)
    tol = U * (len(dy) / 1024 + 75) * mag
    assert (off <= tol).all(), (off / np.maximum(tol, 1e-300)).max()


def backward(q, rng, rows, cols, dtype, dres=True, dgamma=True, accumulate=False, gamma="bf16", ld=None, offset=0,
             inplace=None):
    import torch

    dy = make(rng, rows, cols, dtype, 1e-3, ld, offset)
    h = make(rng, rows, cols, dtype, 2.0, ld, offset)
    dr = make(rng, rows, cols, dtype, 1e-3, ld, offset) if dres else None
    w = weights(rng, cols, gamma)
    rstd = to_dev(oracle.norm.rstd(to_np(h), EPS).astype(np.float32))
    dyv, drv = to_np(dy).copy(), to_np(dr).copy() if dres else None
    dx = {"dy": dy, "dres": dr}.get(inplace)
    if dx is None:
        dx = make(rng, rows, cols, dtype, 1.0, ld, offset)
    dg = start = None
    if dgamma:
        dg = to_dev(rng.standard_normal(cols).astype(np.float32))
        start = to_np(dg).copy() if accumulate else None
    nbytes = q.qsg_rmsnorm_bwd_workspace(rows, cols)
    guard = torch.full((nbytes + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    q.qsg_rmsnorm_bwd(dy, h, w, rstd, dx, dres=dr, dgamma=dg, accumulate=accumulate, workspace=guard[:nbytes])
    torch.cuda.synchronize()
    assert (guard[nbytes:] == 0xA5).all(), "a byte after the workspace was written"
    close_dx(dx, dyv, to_np(h), to_np(rstd), to_np(w), drv, dtype)
    if dgamma:
        close_dgamma(dg, dyv, to_np(h), to_np(rstd), start)
    return dx, dg


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", [
    (1, 1), (1, 8), (3, 7), (5, 64), (130, 500), (1300, 519), (7, 520), (64, 2048), (33, 2055), (40, 4096), (9, 4103),
    (20, 8192), (6, 8195), (5, 16384), (4, 16391), (3, 16392), (2, 20005), (2500, 264), (1100, 1040),
    (400, 3001), (1290, 2600), (1301, 1100), (1311, 4100), (390, 5003)])
def test_backward(q, dtype, rows, cols):
    rng = np.random.default_rng([rows, cols])
    backward(q, rng, rows, cols, dtype)
    backward(q, rng, rows, cols, dtype, dres=False, accumulate=True, gamma="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_views_and_aliases(q, dtype):
    rng = np.random.default_rng(21)
    for cols in (264, 1111):
        backward(q, rng, 37, cols, dtype, ld=cols + 5, offset=1)
        backward(q, rng, 37, cols, dtype, ld=cols + 8, inplace="dy")
        backward(q, rng, 37, cols, dtype, ld=cols + 1, inplace="dres")
        backward(q, rng, 37, cols, dtype, dgamma=False)
    backward(q, rng, 3, 17000, dtype, inplace="dy")


def test_backward_of_no_rows_clears_dgamma(q):
    import torch

    e = torch.empty((0, 16), device="cuda")
    dg = torch.ones(16, device="cuda")
    q.qsg_rmsnorm_bwd(e, e, torch.ones(16, device="cuda"), torch.empty(0, device="cuda"), e, dgamma=dg, accumulate=True)
    assert (dg == 1).all()
    q.qsg_rmsnorm_bwd(e, e, torch.ones(16, device="cuda"), torch.empty(0, device="cuda"), e, dgamma=dg)
    assert (dg == 0).all()


def test_backward_is_the_gradient_of_the_forward(q):
    """Differences of the library's own fp32 forward along random directions."""
    import torch

    rng = np.random.default_rng(31)
    rows, cols = 6, 200
    h, w, dy = make(rng, rows, cols, "f32"), weights(rng, cols, "f32"), make(rng, rows, cols, "f32")
    y, rstd = torch.empty_like(h), torch.empty(rows, device="cuda")

    def loss(h, w):
        q.qsg_rmsnorm_quantize(h, w, EPS, rstd=rstd, y=y)
        return (dy.double() * y.double()).sum().item()

    loss(h, w)
    dx, dg = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    q.qsg_rmsnorm_bwd(dy, h, w, rstd, dx, dgamma=dg, workspace=ws)
    for _ in range(4):
        d, e = make(rng, rows, cols, "f32"), make(rng, 1, cols, "f32").view(-1)
        step = 2.0 ** -9
        slope = (loss(h + step * d, w + step * e) - loss(h - step * d, w - step * e)) / (2 * step)
        want = (dx.double() * d.double()).sum().item() + (dg.double() * e.double()).sum().item()
        # binary32 y: 3 roundings of each of the two losses; and the third derivative's step^2
        scale = (dy.double() * y.double()).abs().sum().item()
        assert abs(slope - want) <= 2 * 4 * U * scale / (2 * step) + step ** 2 * 10 * scale


def test_same_bits_twice_and_on_another_stream(q):
    import torch

    rng = np.random.default_rng(41)
    rows, cols = 1500, 1032
    dy, h, w = make(rng, rows, cols, "bf16"), make(rng, rows, cols, "bf16"), weights(rng, cols, "bf16")
    rstd = to_dev(oracle.norm.rstd(to_np(h), EPS).astype(np.float32))
    got = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        stream.wait_stream(torch.cuda.current_stream())
        dx, dg = torch.empty_like(dy), torch.empty(cols, device="cuda")
        ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        q.qsg_rmsnorm_bwd(dy, h, w, rstd, dx, dgamma=dg, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        got.append((dx, dg))
    for dx, dg in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dg, got[0][1])
