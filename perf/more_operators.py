"""Cases, plain forms and 64-bit values of an MLP in 8-bit integers.

Five operators: the quantization to INT8 with a scale for each token (and, in a
transposed copy, for each channel) ("quant"), the product of two such matrices
("gemm"), the gated activation a = silu(g) u that keeps g and u in 8 bits for
backward ("act_fwd"), its backward pass from those ("act_bwd"), and the weight
gradient from an input kept in 8 bits ("wgrad").  "mlp" is a forward pass
through the MLP in INT8, as a server makes it.  With ``own`` false, ``run``
computes them in elementary torch operations; with ``own`` true it calls the
library.
"""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
BLOCK = 128                       # elements that share a scale of the kept activations
TINY = 2.0 ** -126                # smallest scale
MOST_QUANT = 32768 * 4096         # elements of a drawn case
MOST_ACT = 16384 * 14336          # outputs of a drawn case
MOST_PRODUCTS = 32768 * 4096 * 4096
MOST_WEIGHTS = 3 * 14336 * 4096   # of a drawn MLP


def listed():
    return [
        # the activations of a 4096-hidden training step: one scale per token
        dict(name="quant_train", op="quant", rows=32768, cols=4096, dtype=BF16, t=False),
        # fp32 master weights of its larger Linear: row-wise for fprop, column-wise (transposed) for dgrad
        dict(name="quant_weights_f32", op="quant", rows=14336, cols=4096, dtype=F32, t=True),
        # a ragged prefill through a Linear with a bias
        dict(name="gemm_prefill_bias", op="gemm", m=1021, n=4096, k=4096, out=BF16, bias=True),
        # fprop of the training step
        dict(name="gemm_train", op="gemm", m=32768, n=4096, k=4096, out=BF16, bias=False),
        # the activation of a short ragged fp32 micro-batch
        dict(name="act_fwd_f32_odd", op="act_fwd", rows=333, cols=1111, dtype=F32),
        # the activation of the 14336-wide MLP in training
        dict(name="act_fwd_train", op="act_fwd", rows=16384, cols=14336, dtype=BF16),
        # backward of a short ragged fp32 micro-batch, without the recomputed activation
        dict(name="act_bwd_f32_odd", op="act_bwd", rows=333, cols=1111, dtype=F32, again=False),
        # backward in training, with the activation recomputed for the down projection's weight gradient
        dict(name="act_bwd_train", op="act_bwd", rows=16384, cols=14336, dtype=BF16, again=True),
        # a ragged micro-batch's weight gradient
        dict(name="wgrad_odd", op="wgrad", t=777, n=1000, k=1111, out=BF16),
        # the 4096x4096 Linear's weight gradient into an fp32 main gradient
        dict(name="wgrad_train", op="wgrad", t=32768, n=4096, k=4096, out=F32),
        # one decoded token through the 14336-wide MLP
        dict(name="mlp_token", op="mlp", rows=1, hidden=4096, ffn=14336),
        # a ragged decode batch through it
        dict(name="mlp_batch", op="mlp", rows=61, hidden=4096, ffn=14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "act_fwd", "act_bwd", "wgrad", "mlp"])
    dtype = rng.choice([BF16, BF16, BF16, F32])

    def size(lo, hi):
        """Half of all sizes are multiples of 128, as a model's widths are."""
        n = _log(rng, lo, hi)
        return max(BLOCK, n // BLOCK * BLOCK) if rng.random() < 0.5 else n

    if op == "quant":
        cols = size(64, 16384)
        return dict(op=op, rows=min(_log(rng, 1, 32768), MOST_QUANT // cols // (2 if dtype == F32 else 1)), cols=cols,
                    dtype=dtype, t=rng.random() < 0.4)
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 32768), size(64, 14336), size(64, 14336)
            if m * n * k <= MOST_PRODUCTS:
                return dict(op=op, m=m, n=n, k=k, out=dtype, bias=rng.random() < 0.4)
    if op in ("act_fwd", "act_bwd"):
        cols = size(64, 18432)
        c = dict(op=op, rows=min(_log(rng, 1, 32768), MOST_ACT // cols // (2 if dtype == F32 else 1)), cols=cols,
                 dtype=dtype)
        if op == "act_bwd":
            c["again"] = rng.random() < 0.5
        return c
    if op == "wgrad":
        while True:
            t, n, k = _log(rng, 1, 32768), size(64, 14336), size(64, 14336)
            if t * n * k <= MOST_PRODUCTS:
                return dict(op=op, t=t, n=n, k=k, out=dtype)
    while True:
        hidden, ffn = size(256, 7168), size(256, 18432)
        if hidden * ffn * 3 <= MOST_WEIGHTS:
            return dict(op=op, rows=_log(rng, 1, 1024), hidden=hidden, ffn=ffn)


def _type(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    def stream(rows, cols, dtype):
        """Activations with a few channels far larger than the rest."""
        x = normal(rows, cols)
        x[:, torch.randint(0, cols, (max(1, cols // 100),), generator=g, device=dev)] *= 20.0
        return x.to(dtype)

    def empty(*shape, dtype):
        return torch.empty(*shape, device=dev, dtype=dtype)

    op, s = case["op"], {"case": case}
    if op == "quant":
        R, C = case["rows"], case["cols"]
        s["x"] = normal(R, C, std=0.02) if case["t"] else stream(R, C, _type(case["dtype"]))
        s["x"] = s["x"].to(_type(case["dtype"]))
        s["q"], s["s"] = empty(R, C, dtype=torch.int8), empty(R, dtype=torch.float32)
        if case["t"]:
            s["qt"], s["st"] = empty(C, R, dtype=torch.int8), empty(C, dtype=torch.float32)
            if own:
                import quantize_scaled_gemm_amd as q

                s["workspace"] = torch.empty(q.qsg_quantize_int8_workspace(R, C), dtype=torch.uint8, device=dev)
    elif op == "gemm":
        M, N, K = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _quantize(stream(M, K, torch.bfloat16))
        s["b"], s["sb"] = _quantize(normal(N, K, std=0.02))
        s["bias"] = normal(N, std=0.1, dtype=torch.bfloat16) if case["bias"] else None
        s["c"] = empty(M, N, dtype=_type(case["out"]))
    elif op == "act_fwd":
        R, C, dt = case["rows"], case["cols"], _type(case["dtype"])
        s["gu"] = stream(R, 2 * C, dt)
        s["a"] = empty(R, C, dtype=dt)
        s["ck"], s["cs"] = empty(R, 2 * C, dtype=torch.int8), empty(R, 2 * -(-C // BLOCK), dtype=torch.float32)
    elif op == "act_bwd":
        R, C, dt = case["rows"], case["cols"], _type(case["dtype"])
        s["ck"], s["cs"] = _keep(stream(R, 2 * C, dt))
        s["da"] = normal(R, C, std=1e-3, dtype=dt)
        s["dgu"] = empty(R, 2 * C, dtype=dt)
        s["a"] = empty(R, C, dtype=dt) if case["again"] else None
    elif op == "wgrad":
        T, N, K = case["t"], case["n"], case["k"]
        s["q"], s["s"] = _quantize(stream(T, K, torch.bfloat16))
        s["dy"] = normal(T, N, std=1e-3, dtype=torch.bfloat16)
        s["c"] = empty(N, K, dtype=_type(case["out"]))
    else:
        R, H, F = case["rows"], case["hidden"], case["ffn"]
        s["x"] = stream(R, H, torch.bfloat16)
        s["w1"], s["s1"] = _quantize(normal(2 * F, H, std=H ** -0.5))
        s["w2"], s["s2"] = _quantize(normal(H, F, std=F ** -0.5))
        s["q"], s["s"] = empty(R, H, dtype=torch.int8), empty(R, dtype=torch.float32)
        s["gu"] = empty(R, 2 * F, dtype=torch.bfloat16)
        s["aq"], s["as"] = empty(R, F, dtype=torch.int8), empty(R, dtype=torch.float32)
        s["y"] = empty(R, H, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _scale(amax):
    """The scale of a maximum: amax / 127, a tensor in the divisor's place so that it is a division."""
    s = (amax / torch.full_like(amax, 127.0)).clamp(min=TINY)
    return torch.where(amax == 0, torch.ones_like(s), s)


def _codes(x, s):
    return torch.round(x * torch.reciprocal(s)).clamp(-127, 127).to(torch.int8)


def _quantize(x):
    """(codes, scales) of the rows of x."""
    x = x.float()
    s = _scale(x.abs().amax(dim=1))
    return _codes(x, s.unsqueeze(1)), s


def _keep(gu):
    """(codes, scales) of g and u in blocks along the row; a last short block is a block."""
    R, C = gu.shape[0], gu.shape[1] // 2
    nb = -(-C // BLOCK)
    x = torch.nn.functional.pad(gu.float().view(R, 2, C), (0, nb * BLOCK - C)).view(R, 2, nb, BLOCK)
    s = _scale(x.abs().amax(dim=-1))
    q = _codes(x, s.unsqueeze(-1)).view(R, 2, nb * BLOCK)[:, :, :C]
    return q.reshape(R, 2 * C), s.view(R, 2 * nb)


def _kept(ck, cs):
    """g and u as the kept codes stand for them."""
    R, C = ck.shape[0], ck.shape[1] // 2
    nb = cs.shape[1] // 2
    s = cs.view(R, 2, nb, 1).expand(R, 2, nb, BLOCK).reshape(R, 2, nb * BLOCK)[:, :, :C]
    x = ck.view(R, 2, C).float() * s
    return x[:, 0], x[:, 1]


def _product(a, sa, b, sb, bias, dtype):
    c = (a.float() @ b.float().t()) * sa.unsqueeze(1) * sb
    if bias is not None:
        c = c + bias.float()
    return c.to(dtype)


def _act(gu):
    C = gu.shape[1] // 2
    g, u = gu[:, :C].float(), gu[:, C:].float()
    return g / (1.0 + torch.exp(-g)) * u


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        out = dict(zip(("q", "s"), _quantize(s["x"])))
        if case["t"]:
            out |= dict(zip(("qt", "st"), _quantize(s["x"].t().contiguous())))
        return out
    if op == "gemm":
        return {"c": _product(s["a"], s["sa"], s["b"], s["sb"], s["bias"], _type(case["out"]))}
    if op == "act_fwd":
        ck, cs = _keep(s["gu"])
        return {"a": _act(s["gu"]).to(s["gu"].dtype), "ck": ck, "cs": cs}
    if op == "act_bwd":
        g, u = _kept(s["ck"], s["cs"])
        da, dt = s["da"].float(), s["da"].dtype
        sig = 1.0 / (1.0 + torch.exp(-g))
        silu = g * sig
        out = {"dgu": torch.cat([da * u * (sig * (1.0 + g * (1.0 - sig))), da * silu], dim=1).to(dt)}
        if case["again"]:
            out["a"] = (silu * u).to(dt)
        return out
    if op == "wgrad":
        # the operand that the codes stand for is a bf16 matrix, as the tensor that was quantized
        x = (s["q"].float() * s["s"].unsqueeze(1)).to(torch.bfloat16)
        return {"c": (s["dy"].float().t() @ x.float()).to(_type(case["out"]))}
    q, sx = _quantize(s["x"])
    gu = _product(q, sx, s["w1"], s["s1"], None, torch.bfloat16)
    q, sx = _quantize(_act(gu))
    return {"y": _product(q, sx, s["w2"], s["s2"], None, torch.bfloat16)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import quantize_scaled_gemm_amd as q

    case = s["case"]
    op = case["op"]
    if op == "quant":
        if case["t"]:
            q.qsg_quantize_int8(s["x"], q=s["q"], s=s["s"], qt=s["qt"], st=s["st"], workspace=s["workspace"])
            return {k: s[k] for k in ("q", "s", "qt", "st")}
        q.qsg_quantize_int8(s["x"], q=s["q"], s=s["s"])
        return {"q": s["q"], "s": s["s"]}
    if op == "gemm":
        q.qsg_gemm_int8(s["a"], s["sa"], s["b"], s["sb"], s["c"], bias=s["bias"])
        return {"c": s["c"]}
    if op == "act_fwd":
        q.qsg_swiglu_int8_store_fwd(s["gu"], a=s["a"], ck=s["ck"], cs=s["cs"])
        return {"a": s["a"], "ck": s["ck"], "cs": s["cs"]}
    if op == "act_bwd":
        q.qsg_swiglu_int8_store_bwd(s["da"], s["ck"], s["cs"], s["dgu"], a=s["a"])
        return {"dgu": s["dgu"], "a": s["a"]} if case["again"] else {"dgu": s["dgu"]}
    if op == "wgrad":
        q.qsg_wgrad_int8(s["dy"], s["q"], s["s"], s["c"])
        return {"c": s["c"]}
    q.qsg_quantize_int8(s["x"], q=s["q"], s=s["s"])
    q.qsg_gemm_int8(s["q"], s["s"], s["w1"], s["s1"], s["gu"])
    q.qsg_swiglu_int8_store_fwd(s["gu"], aq=s["aq"], sa=s["as"])
    q.qsg_gemm_int8(s["aq"], s["as"], s["w2"], s["s2"], s["y"])
    return {"y": s["y"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    b = 2 if case.get("dtype", case.get("out")) == BF16 else 4
    if op == "quant":
        R, C = case["rows"], case["cols"]
        copies = 1 + case["t"]
        return {"bytes": R * C * (b + copies) + 4 * R + 4 * C * case["t"], "flops": R * C * (2 + 2 * copies)}
    if op == "gemm":
        M, N, K = case["m"], case["n"], case["k"]
        return {"bytes": (M + N) * (K + 4) + M * N * b + 2 * N * case["bias"], "flops": 2 * M * N * K}
    if op in ("act_fwd", "act_bwd"):
        R, C = case["rows"], case["cols"]
        n, scales = R * C, 8 * R * -(-C // BLOCK)
        if op == "act_fwd":
            return {"bytes": n * (3 * b + 2) + scales, "flops": 14 * n}
        return {"bytes": n * (3 * b + 2 + b * case["again"]) + scales, "flops": 14 * n}
    if op == "wgrad":
        T, N, K = case["t"], case["n"], case["k"]
        return {"bytes": T * (2 * N + K + 4) + N * K * b, "flops": 2 * T * N * K}
    R, H, F = case["rows"], case["hidden"], case["ffn"]
    return {"bytes": 3 * H * F + 4 * (2 * F + H) + 4 * R * H, "flops": 6 * R * H * F}


# ---------------------------------------------------------------------------
# 64-bit values
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op, wide = prepare(case, seed), case["op"], torch.float64

    def coded(x, dim):
        """Codes and scales along a dimension: the scale, its reciprocal and the product with it are binary32 values by
        definition, and the codes follow from them alone."""
        top = x.abs().max(dim=dim, keepdim=True).values
        step = torch.where(top == 0, torch.ones_like(top), torch.maximum((top / 127).float().to(wide),
                                                                         torch.full_like(top, 2.0 ** -126)))
        inv = (1 / step).float().to(wide)
        code = torch.minimum(torch.maximum(torch.round((x * inv).float()), torch.tensor(-127.0, device=x.device)),
                             torch.tensor(127.0, device=x.device))
        return code.to(torch.int8), torch.where(top == 0, torch.ones_like(top), top / 127)

    if op == "quant":
        x = s["x"].to(wide)
        out = {}
        out["q"], step = coded(x, 1)
        out["s"] = step.reshape(-1)
        if case["t"]:
            code, step = coded(x, 0)
            out["qt"], out["st"] = code.t().contiguous(), step.reshape(-1)
        return out
    if op == "gemm":
        c = s["a"].to(wide) @ s["b"].to(wide).t()
        c *= torch.outer(s["sa"].to(wide), s["sb"].to(wide))
        return {"c": c if s["bias"] is None else c + s["bias"].to(wide)}
    if op == "act_fwd":
        C = case["cols"]
        out = {"a": torch.sigmoid(s["gu"][:, :C].to(wide)).mul_(s["gu"][:, :C].to(wide)).mul_(s["gu"][:, C:].to(wide))}
        edges = [(h + k, h + min(k + 128, C)) for h in (0, C) for k in range(0, C, 128)]
        parts = [coded(s["gu"][:, lo:hi].to(wide), 1) for lo, hi in edges]
        out["ck"] = torch.cat([p[0] for p in parts], dim=1)
        out["cs"] = torch.cat([p[1] for p in parts], dim=1)
        return out
    if op == "act_bwd":
        C = case["cols"]
        step = s["cs"].to(wide)
        nb = step.shape[1] // 2
        at = torch.arange(C, device=step.device) // 128
        # a code times its scale is a binary32 value by definition
        g = (s["ck"][:, :C].to(wide) * step[:, at]).float().to(wide)
        u = (s["ck"][:, C:].to(wide) * step[:, nb + at]).float().to(wide)
        sig = torch.sigmoid(g)
        dgu = torch.empty(case["rows"], 2 * C, dtype=wide, device=step.device)
        da = s["da"].to(wide)
        dgu[:, :C] = da * u * (sig + g * sig * torch.sigmoid(-g))
        dgu[:, C:] = da * (g * sig)
        return {"dgu": dgu, "a": g * sig * u} if case["again"] else {"dgu": dgu}
    if op == "wgrad":
        x = (s["q"].to(wide) * s["s"].to(wide)[:, None]).float().to(torch.bfloat16).to(wide)
        return {"c": s["dy"].to(wide).t().contiguous() @ x}
    q, step = coded(s["x"].to(wide), 1)
    # the matrix between the two products is stored in bf16 by definition
    gu = (q.to(wide) @ s["w1"].to(wide).t() * torch.outer(step.reshape(-1), s["s1"].to(wide))).to(torch.bfloat16).to(wide)
    g, u = gu[:, :case["ffn"]], gu[:, case["ffn"]:]
    q, step = coded((g * torch.sigmoid(g) * u).float().to(wide), 1)
    return {"y": q.to(wide) @ s["w2"].to(wide).t() * torch.outer(step.reshape(-1), s["s2"].to(wide))}
