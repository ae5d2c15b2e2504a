"""The forms of the norm calls that a shape, a recipe or a missing output
chooses, each against the 64-bit oracle: column-wise copies alone, no rstd,
every way that a row is held with more rows than its single-row form takes,
and the loops of the kernels whose workgroups take several rows in turn."""

import numpy as np
import pytest

import oracle
from helpers import to_dev, to_np
from test_gpu_norm import EPS, HALF, U, longest, make, quantizers, same, torch_type, weights
from test_gpu_norm_sums import bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantize_scaled_gemm_amd as q

    q.load_library()
    return q


def forward(q, rng, rows, cols, dtype, recipe, row=True, col=True, rstd=True, residual=True, ld=None, offset=0,
            fmt="e4m3", rule="ceil"):
    """One call with the copies that are asked for, checked against the oracle."""
    import torch

    codes = {"mx": q.MXFP8, "1x128": q.BLOCK_1X128, "delayed": q.DELAYED, "tensorwise": q.TENSORWISE}
    x = make(rng, rows, cols, dtype, 1.0, ld, offset)
    r = make(rng, rows, cols, dtype, 2.0, ld, offset) if residual else None
    w = weights(rng, cols, "f32")
    hv = to_np(x) if r is None else to_np(torch.from_numpy(to_np(x) + to_np(r)).to(x.dtype))
    u8 = dict(dtype=torch.uint8, device="cuda")
    o = dict(h=torch.empty_like(x) if residual else None, rstd=torch.empty(rows, device="cuda") if rstd else None)
    guard = torch.full((2, rows * cols + 2), 0xA5, **u8)
    scale = None
    if row:
        o["q"] = guard[0, 1:-1].view(rows, cols)
    if col:
        o["qt"] = guard[1, 1:-1].view(cols, rows)
    if recipe == "mx":
        o["s"] = torch.empty((rows, cols // 32), **u8) if row else None
        o["st"] = torch.empty((cols, rows // 32), **u8) if col else None
    elif recipe == "1x128":
        o["s"] = torch.empty((rows, cols // 128), device="cuda") if row else None
        o["st"] = torch.empty((cols, rows // 128), device="cuda") if col else None
    elif recipe == "tensorwise":
        o["s"] = torch.empty(3, device="cuda")
    else:
        scale = torch.full((1,), 40.0, device="cuda")
        o["amax_out"] = torch.full((1,), -1.0, device="cuda")
    q.qsg_rmsnorm_quantize(x, w, EPS, codes[recipe], q.FMT[fmt], residual=r, scale=scale,
                           mx_rule=q.MX_CEIL if rule == "ceil" else q.MX_OCP_FLOOR, **o)
    torch.cuda.synchronize()
    if residual:
        same(o["h"], hv, "h")
    if not rstd:
        # what the same call gives when asked for it
        o["rstd"] = torch.empty(rows, device="cuda")
        q.qsg_rmsnorm_quantize(x, w, EPS, residual=r, h=o["h"], rstd=o["rstd"], y=torch.empty((rows, cols), dtype=x.dtype, device="cuda"))
    want = oracle.norm.rstd(hv, EPS)
    assert (np.abs(to_np(o["rstd"]).astype(np.float64) - want) <= (longest(cols) / 2 + 5) * U * want).all()
    y = oracle.norm.normed_f32(hv, to_np(o["rstd"]), to_np(w))
    wq, ws, wqt, wst, wamax = quantizers(recipe, y, fmt, 0, rule, np.float32(40.0))
    if row:
        same(o["q"], wq, "q")
    if row or recipe == "tensorwise":
        if ws is not None:
            same(o["s"], ws, "s")
    if col:
        same(o["qt"], wqt, "qt")
        if wst is not None:
            same(o["st"], wst, "st")
    if wamax is not None:
        same(o["amax_out"], np.float32([wamax]), "amax")
    g = guard.cpu().numpy()
    assert (g[:, 0] == 0xA5).all() and (g[:, -1] == 0xA5).all(), "a byte outside q or qt was written"
    assert row or (g[0] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("recipe, rows, cols", [
    ("delayed", 65, 131), ("delayed", 300, 2049), ("delayed", 1, 1), ("delayed", 130, 63), ("delayed", 3, 20011),
    ("mx", 32, 7), ("mx", 96, 45), ("mx", 160, 101), ("mx", 64, 16400), ("mx", 128, 64),
    ("1x128", 128, 5), ("1x128", 256, 200), ("1x128", 384, 65),
    ("tensorwise", 200, 300), ("tensorwise", 129, 31), ("tensorwise", 1, 7)])
def test_column_copy_alone(q, dtype, recipe, rows, cols):
    """Columns in any number, blocks running down the rows alone."""
    rng = np.random.default_rng([rows, cols])
    forward(q, rng, rows, cols, dtype, recipe, row=False)
    forward(q, rng, rows, cols, dtype, recipe, row=False, residual=False, ld=cols + 3, offset=1, fmt="e5m2")
    if recipe == "mx":
        forward(q, rng, rows, cols, dtype, recipe, row=False, rule="ocp")


@pytest.mark.parametrize("recipe, rows, cols", [("mx", 5, 256), ("mx", 300, 4096), ("1x128", 2, 7168),
                                                ("delayed", 40, 515), ("delayed", 2, 20011)])
def test_without_rstd(q, recipe, rows, cols):
    for residual in (False, True):
        forward(q, np.random.default_rng(1), rows, cols, "bf16", recipe, col=False, rstd=False, residual=residual)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("recipe, rows, cols", [
    # threads a row x chunks a thread, without an amax: 16 x 1, 16 x 2, 64 x 1, 64 x 2, 256 x 1, 2, 4, 512 x 4, twice read
    ("mx", 320, 128), ("mx", 320, 256), ("1x128", 384, 512), ("mx", 288, 1024), ("1x128", 384, 2048), ("mx", 288, 4096),
    ("1x128", 384, 7168), ("mx", 320, 5024), ("mx", 288, 8224), ("1x128", 384, 16384), ("mx", 288, 16416),
    # with one
    ("tensorwise", 257, 8224), ("delayed", 260, 16384), ("delayed", 300, 8224), ("tensorwise", 300, 16411)])
def test_more_rows_than_compute_units(q, dtype, recipe, rows, cols):
    """From 257 rows on a row no longer has a workgroup of 1024 threads."""
    forward(q, np.random.default_rng([rows, cols]), rows, cols, dtype, recipe)


@pytest.mark.parametrize("rows, cols", [(16500, 40), (16390, 200), (4200, 300), (4200, 1000), (1100, 8208), (1030, 16392)])
def test_amax_workgroups_that_take_rows_in_turn(q, rows, cols):
    """Rows beyond the persistent grid of a launch with an amax output."""
    forward(q, np.random.default_rng(cols), rows, cols, "bf16", "delayed", col=False)


def test_rows_beyond_the_largest_grid(q):
    """More than 2^20 workgroups of 16 rows: the last rows are those of a call on
    them alone."""
    import torch

    rows, cols, tail = (1 << 24) + 50, 5, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    got = []
    for v in (x, x[-tail:]):
        y, rstd = torch.empty_like(v), torch.empty(v.shape[0], device="cuda")
        q.qsg_rmsnorm_quantize(v, w, EPS, rstd=rstd, y=y)
        got.append((y[-tail:], rstd[-tail:]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def backward(q, rows, cols, dtype, dres, accumulate, sample=None):
    """dx of every row (or of some), and dgamma."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(rows + cols)

    def normal(std, *shape, kind=torch_type(dtype)):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(kind)

    dy, h = normal(1e-3, rows, cols), normal(2.0, rows, cols)
    dr = normal(1e-3, rows, cols) if dres else None
    w = 1 + normal(0.1, cols, kind=torch.float32)
    rstd = torch.rand(rows, generator=g, device="cuda") + 0.3
    dg = normal(1.0, cols, kind=torch.float32)
    start = to_np(dg).astype(np.float64) if accumulate else np.zeros(cols)
    dx = torch.empty_like(dy)
    ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    q.qsg_rmsnorm_bwd(dy, h, w, rstd, dx, dres=dr, dgamma=dg, accumulate=accumulate, workspace=ws)
    at = np.arange(rows) if sample is None else np.asarray(sample)
    pick = to_dev(at)
    a = [to_np(t[pick]) if t is not None else None for t in (dy, h, rstd, dr, dx)]
    ref, _ = oracle.norm.norm_bwd(a[0], a[1], a[2], to_np(w), a[3])
    off = np.abs(a[4].astype(np.float64) - ref)
    most = oracle.norm.norm_bwd_bound(a[0], a[1], a[2], to_np(w), a[3], longest(cols), HALF[dtype])
    assert (off <= most).all(), f"dx: {(off / np.maximum(most, 1e-300)).max():.3g} times its bound"
    ref, mag = np.zeros(cols), np.zeros(cols)
    for part in torch.arange(rows, device="cuda").split(1024):
        term = dy[part].double() * h[part].double() * rstd[part].double()[:, None]
        ref += to_np(term.sum(0))
        mag += to_np(term.abs().sum(0))
    ref, mag = ref + start, mag + np.abs(start)
    off = np.abs(to_np(dg).astype(np.float64) - ref)
    assert (off <= bound(rows, cols, mag, ref)).all(), "dgamma"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", [
    (9000, 40), (9000, 200), (5000, 500), (17000, 600), (3000, 1111), (1100, 4100), (1601, 5000), (600, 9000),
    (300, 16500), (140, 40000)])
def test_backward_groups_that_take_rows_in_turn(q, dtype, rows, cols):
    """More rows than groups in every form: 16 lanes, a wave, one, two and four
    rows a workgroup, 1024 threads a row, and rows in pieces."""
    for dres, accumulate in ((True, False), (False, True)):
        backward(q, rows, cols, dtype, dres, accumulate)


def test_backward_dots_that_take_rows_in_turn(q):
    """More than 4096 rows beyond the registers; some rows' dx, all of dgamma."""
    backward(q, 4100, 16392, "bf16", True, False, sample=[0, 1, 127, 128, 2050, 4094, 4095, 4096, 4097, 4099])
