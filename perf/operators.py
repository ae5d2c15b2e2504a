"""Cases, plain forms and 64-bit values of the operators around an FP8 Linear.

Three operators: the residual addition with an RMS norm and an FP8 output
("norm"), its backward pass ("norm_bwd"), and the global norm of many gradient
tensors with clipping ("clip").  With ``own`` false, ``run`` computes them in
elementary torch operations; with ``own`` true it calls the library.
"""

import math

import torch

own = False

EPS = 1e-5
MAX_NORM = 1.0
BF16, F32 = "bf16", "f32"
E4M3_MAX = 448.0
MOST_ELEMENTS = 32768 * 4096  # of a drawn norm case
MOST_GRADS = 300_000_000      # of a drawn clip case


def listed():
    return [
        # one decoded token of a 4096-hidden model under MXFP8
        dict(name="norm_token_mx", op="norm", rows=1, cols=4096, dtype=BF16, recipe="mx", residual=True, t=False,
             y=False),
        # a decode batch of a 7168-hidden model with 1x128 blocks
        dict(name="norm_batch_1x128", op="norm", rows=64, cols=7168, dtype=BF16, recipe="1x128", residual=True,
             t=False, y=False),
        # a ragged prefill with a calibrated scale; the bf16 output feeds a layer that stays in bf16
        dict(name="norm_prefill_delayed_y", op="norm", rows=1021, cols=4096, dtype=BF16, recipe="delayed",
             residual=True, t=False, y=True),
        # fp32 activations of odd sizes, current scaling, first norm of a model (no residual yet)
        dict(name="norm_f32_tensorwise_odd", op="norm", rows=1003, cols=1111, dtype=F32, recipe="tensorwise",
             residual=False, t=True, y=False),
        # the delayed-scaling training step's activations
        dict(name="norm_train_delayed", op="norm", rows=8192, cols=4096, dtype=BF16, recipe="delayed", residual=True,
             t=True, y=False),
        # the 4096-hidden training step's activations, MXFP8
        dict(name="norm_train_mx", op="norm", rows=32768, cols=4096, dtype=BF16, recipe="mx", residual=True, t=True,
             y=False),
        # the 7168-hidden training step's activations, 1x128 blocks
        dict(name="norm_train_1x128", op="norm", rows=16384, cols=7168, dtype=BF16, recipe="1x128", residual=True,
             t=True, y=False),
        # backward of a short ragged fp32 micro-batch
        dict(name="bwd_f32_odd", op="norm_bwd", rows=333, cols=1111, dtype=F32, residual=True),
        # backward of the delayed step's activations at the model's first norm
        dict(name="bwd_8192x4096", op="norm_bwd", rows=8192, cols=4096, dtype=BF16, residual=False),
        # backward of the 7168-hidden step's activations
        dict(name="bwd_16384x7168", op="norm_bwd", rows=16384, cols=7168, dtype=BF16, residual=True),
        # the gradients of a small model, odd sizes, bf16
        dict(name="clip_small_bf16", op="clip", layers=6, hidden=257, ffn=1001, dtype=BF16),
        # fp32 main gradients of four 4096-hidden layers
        dict(name="clip_main_f32", op="clip", layers=4, hidden=4096, ffn=14336, dtype=F32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "clip"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op == "clip":
        while True:
            c = dict(op=op, layers=_log(rng, 1, 24), hidden=_log(rng, 32, 4096), ffn=_log(rng, 64, 14336), dtype=dtype)
            if sum(math.prod(s) for s in _shapes(c)) <= MOST_GRADS:
                return c
    most = MOST_ELEMENTS // (2 if dtype == F32 else 1)
    rows, cols = _log(rng, 1, 32768), _log(rng, 128, 16384)
    if op == "norm_bwd":
        rows = min(rows, most // cols)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7)
    recipe = rng.choice(["mx", "1x128", "delayed", "tensorwise"])
    t = rng.random() < 0.5
    block = {"mx": 32, "1x128": 128}.get(recipe, 1)
    cols = max(block, cols // block * block)
    if rng.random() < 0.5:
        cols = max(128, cols // 128 * 128)
    rows = min(rows, most // cols)
    if t:
        rows = max(block, rows // block * block)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, recipe=recipe, residual=rng.random() < 0.7, t=t,
                y=rng.random() < 0.25)


def _shapes(case):
    """The gradient tensors: per layer a norm weight and the two Linear weights."""
    h, f = case["hidden"], case["ffn"]
    return [(h,), (h, h), (f, h)] * case["layers"]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": case}
    if case["op"] == "clip":
        shapes = _shapes(case)
        s["grads"] = [normal(*sh, std=1e-3 * (1 + i % 3)) for i, sh in enumerate(shapes)]
        # the clipped gradients go into the optimizer's flat buffer, each tensor starting at a multiple of 64 elements
        starts, at = [], 0
        for sh in shapes:
            starts.append(at)
            at += (math.prod(sh) + 63) // 64 * 64
        s["flat"] = torch.zeros(at, device=dev, dtype=dt)
        s["outs"] = [s["flat"][a:a + math.prod(sh)].view(sh) for a, sh in zip(starts, shapes)]
        s["norm"] = torch.zeros(1, device=dev)
        s["sumsq"] = torch.zeros(1, device=dev, dtype=torch.float64)
        if own:
            import quantize_scaled_gemm_amd as q

            s["plan"] = q.qsg_grad_plan(s["grads"], s["outs"])
            s["workspace"] = torch.empty(q.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        return s
    R, C = case["rows"], case["cols"]
    s["gamma"] = 1 + normal(C, std=0.1, dtype=torch.float32)
    s["gamma"] = s["gamma"].to(dt)
    # a residual stream with a few channels far larger than the rest
    channel = torch.ones(C, device=dev)
    channel[torch.randint(0, C, (max(1, C // 100),), generator=g, device=dev)] = 20.0
    if case["op"] == "norm":
        s["x"] = normal(R, C)
        s["r"] = (normal(R, C, std=2.0, dtype=torch.float32) * channel).to(dt) if case["residual"] else None
        s["h"] = torch.empty(R, C, device=dev, dtype=dt) if case["residual"] else None
        s["rstd"] = torch.empty(R, device=dev)
        s["y"] = torch.empty(R, C, device=dev, dtype=dt) if case["y"] else None
        u8 = dict(device=dev, dtype=torch.uint8)
        s["q"] = torch.empty(R, C, **u8)
        s["qt"] = torch.empty(C, R, **u8) if case["t"] else None
        s["s"] = s["st"] = s["scale"] = s["amax"] = None
        if case["recipe"] == "mx":
            s["s"] = torch.empty(R, C // 32, **u8)
            s["st"] = torch.empty(C, R // 32, **u8) if case["t"] else None
        elif case["recipe"] == "1x128":
            s["s"] = torch.empty(R, C // 128, device=dev)
            s["st"] = torch.empty(C, R // 128, device=dev) if case["t"] else None
        elif case["recipe"] == "tensorwise":
            s["s"] = torch.empty(3, device=dev)
        else:
            # the scale of the steps before: a little of the tensor saturates
            s["scale"] = torch.full((1,), E4M3_MAX / 8.0, device=dev)
            s["amax"] = torch.empty(1, device=dev)
        return s
    h = (normal(R, C, std=2.0, dtype=torch.float32) * channel).to(dt)
    s["h"] = h
    s["rstd"] = _rstd(h.float())
    s["dy"] = normal(R, C, std=1e-3)
    s["dres"] = normal(R, C, std=1e-3) if case["residual"] else None
    s["dx"] = torch.empty(R, C, device=dev, dtype=dt)
    s["dgamma"] = torch.empty(C, device=dev)
    if own:
        import quantize_scaled_gemm_amd as q

        s["workspace"] = torch.empty(q.qsg_rmsnorm_bwd_workspace(R, C), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rstd(h):
    return 1.0 / torch.sqrt(h.square().mean(dim=-1) + EPS)


def _encode(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _mx(y):
    """(codes, E8M0 scales) of 32-element blocks along the last axis: the smallest power of two without saturation."""
    b = y.view(y.shape[0], -1, 32)
    amax = b.abs().amax(dim=-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-127, 127)
    q = _encode(torch.ldexp(b, -e.unsqueeze(-1))).view(y.shape)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _block(y):
    """(codes, scale_inv) of 128-element blocks along the last axis."""
    b = y.view(y.shape[0], -1, 128)
    amax = b.abs().amax(dim=-1)
    scale = torch.where(amax > 0, E4M3_MAX / amax, torch.ones_like(amax))
    return _encode(b * scale.unsqueeze(-1)).view(y.shape), 1.0 / scale


def _transposed(q):
    return q.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)


def _plain_norm(s):
    case, out = s["case"], {}
    h = s["x"].float()
    if s["r"] is not None:
        out["h"] = (h + s["r"].float()).to(s["x"].dtype)
        h = out["h"].float()
    out["rstd"] = _rstd(h)
    y = h * out["rstd"].unsqueeze(1) * s["gamma"].float()
    if case["y"]:
        out["y"] = y.to(s["x"].dtype)
    if case["recipe"] in ("mx", "1x128"):
        blocked = _mx if case["recipe"] == "mx" else _block
        out["q"], out["s"] = blocked(y)
        if case["t"]:
            out["qt"], out["st"] = blocked(y.t().contiguous())
        return out
    amax = y.abs().amax()
    if case["recipe"] == "tensorwise":
        scale = torch.where(amax > 0, E4M3_MAX / amax, torch.ones_like(amax))
        out["s"] = torch.stack([amax, scale, 1.0 / scale])
    else:
        scale = s["scale"]
        out["amax"] = amax.view(1)
    out["q"] = _encode(y * scale)
    if case["t"]:
        out["qt"] = _transposed(out["q"])
    return out


def _plain_norm_bwd(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"].unsqueeze(1)
    n = h * rstd
    dn = dy * s["gamma"].float()
    dx = rstd * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dy"].dtype), "dgamma": (dy * n).sum(dim=0)}


def _plain_clip(s):
    total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt().float().view(1)
    k = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g * k)
    return {"flat": s["flat"], "norm": norm}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_norm(s):
    import quantize_scaled_gemm_amd as q

    case = s["case"]
    recipe = {"mx": q.MXFP8, "1x128": q.BLOCK_1X128, "delayed": q.DELAYED, "tensorwise": q.TENSORWISE}[case["recipe"]]
    q.qsg_rmsnorm_quantize(s["x"], s["gamma"], EPS, recipe, q.E4M3, residual=s["r"], h=s["h"], rstd=s["rstd"],
                           y=s["y"], q=s["q"], s=s["s"], qt=s["qt"], st=s["st"], scale=s["scale"],
                           amax_out=s["amax"])
    out = {"rstd": s["rstd"], "q": s["q"].view(torch.float8_e4m3fn)}
    if case["residual"]:
        out["h"] = s["h"]
    if case["y"]:
        out["y"] = s["y"]
    if case["t"]:
        out["qt"] = s["qt"].view(torch.float8_e4m3fn)
    if case["recipe"] == "delayed":
        out["amax"] = s["amax"]
    elif case["recipe"] == "mx":
        out["s"] = s["s"].view(torch.float8_e8m0fnu)
        if case["t"]:
            out["st"] = s["st"].view(torch.float8_e8m0fnu)
    else:
        out["s"] = s["s"]
        if case["t"] and case["recipe"] == "1x128":
            out["st"] = s["st"]
    return out


def _own_norm_bwd(s):
    import quantize_scaled_gemm_amd as q

    q.qsg_rmsnorm_bwd(s["dy"], s["h"], s["gamma"], s["rstd"], s["dx"], dres=s["dres"], dgamma=s["dgamma"],
                      workspace=s["workspace"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_clip(s):
    import quantize_scaled_gemm_amd as q

    q.qsg_grad_sumsq(s["plan"], s["sumsq"], s["workspace"])
    q.qsg_grad_clip(s["plan"], s["sumsq"], MAX_NORM, s["norm"])
    return {"flat": s["flat"], "norm": s["norm"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "clip": _own_clip}[op](state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "clip": _plain_clip}[op](state)


def work(case):
    b = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "clip":
        n = sum(math.prod(sh) for sh in _shapes(case))
        return {"bytes": 2 * b * n, "flops": 3 * n}
    R, C = case["rows"], case["cols"]
    n = R * C
    if case["op"] == "norm_bwd":
        return {"bytes": n * b * (3 + case["residual"]) + 4 * R + (b + 4) * C, "flops": 12 * n}
    per = b * (1 + 2 * case["residual"] + case["y"]) + 1 + case["t"]
    copies = 1 + case["t"]
    scales = {"mx": n // 32, "1x128": n // 128 * 4}.get(case["recipe"], 0) * copies
    return {"bytes": n * per + scales + 4 * R + b * C, "flops": (8 + 2 * copies) * n}


# ---------------------------------------------------------------------------
# 64-bit values
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        wide = [g.to(torch.float64).reshape(-1) for g in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(w, w)) for w in wide))
        k = min(1.0, MAX_NORM / (norm + 1e-6))
        flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for w in wide:
            flat[at:at + w.numel()] = w * k
            at += -(-w.numel() // 64) * 64
        return {"flat": flat, "norm": torch.tensor([norm], dtype=torch.float64)}
    w = s["gamma"].to(torch.float64)
    C = case["cols"]
    if case["op"] == "norm_bwd":
        # dx_j = rstd w_j dy_j - rstd^3 h_j / C * sum_k w_k dy_k h_k
        dy, h, rstd = (s[k].to(torch.float64) for k in ("dy", "h", "rstd"))
        inner = (dy * h) @ w
        dx = rstd[:, None] * (dy * w) - h * (rstd ** 3 * inner / C)[:, None]
        if s["dres"] is not None:
            dx += s["dres"].to(torch.float64)
        return {"dx": dx, "dgamma": rstd @ (dy * h)}
    out = {}
    if s["r"] is None:
        h = s["x"].to(torch.float64)
    else:
        # the sum is exact in 64 bits for these inputs; its rounding to the stored type is part of the definition
        out["h"] = s["x"].to(torch.float64) + s["r"].to(torch.float64)
        h = out["h"].to(_dtype(case)).to(torch.float64)
    out["rstd"] = torch.linalg.vector_norm(h, dim=1).square().div(C).add(EPS).pow(-0.5)
    y = h * torch.outer(out["rstd"], w)
    if case["y"]:
        out["y"] = y

    def coded(v):
        return torch.minimum(torch.maximum(v, torch.full_like(v, -448.0)), torch.full_like(v, 448.0))

    def blocks(v, n):
        """Codes (before their rounding) and decode scales of n-element blocks of each row."""
        top = v.reshape(-1, n).abs().max(dim=1).values
        if n == 32:
            step = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(-127, 127))
        else:
            step = top / 448.0
        step = torch.where(top == 0, torch.ones_like(step), step)
        return coded((v.reshape(-1, n) / step[:, None]).reshape(v.shape)), step.reshape(v.shape[0], -1)

    n = {"mx": 32, "1x128": 128}.get(case["recipe"])
    if n:
        out["q"], out["s"] = blocks(y, n)
        if case["t"]:
            out["qt"], out["st"] = blocks(y.t().contiguous(), n)
        if n == 32:
            # a power-of-two scale steps where a block's maximum meets a border: on either side of it by a rounding of
            # the maximum both steps are right, so the exponents have no 64-bit value to be measured against
            out["s"] = None
            if case["t"]:
                out["st"] = None
        return out
    top = float(y.abs().max())
    if case["recipe"] == "tensorwise":
        scale = 448.0 / top if top else 1.0
        out["s"] = torch.tensor([top, scale, 1.0 / scale], dtype=torch.float64)
    else:
        scale = float(s["scale"])
        out["amax"] = torch.tensor([top], dtype=torch.float64)
    out["q"] = coded(y * scale)
    if case["t"]:
        out["qt"] = out["q"].t().contiguous()
    return out
