"""The example's training step part by part, each against 64 bits on the
operands that the step itself made: what quantization costs is left out, so
every part is held to its own roundings, and the norm's gradient to more than
the residual gradient beside it would hide.

With u = 2^-24: a product of K FP8 pairs is exact, and its sum loses at most
2 u of the sum of magnitudes an addition; bf16 results are rounded once (2^-8).
"""

import importlib.util
import os

import numpy as np
import pytest

import oracle
from helpers import ROOT, to_np
from test_gpu_norm import longest
from test_gpu_norm_sums import bound

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T, K, N = 384, 256, 320


@pytest.fixture(scope="module")
def step():
    """Two micro-batches, the main gradients before and after clipping."""
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("prenorm_linear_step", os.path.join(ROOT, "examples", "prenorm_linear_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    gen = torch.Generator(device="cuda").manual_seed(11)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(torch.bfloat16)

    layer = m.PreNormLinear(T, K, N, max_norm=0.25)
    layer.weight.copy_(normal(N, K, std=0.02))
    layer.gamma.copy_(1 + normal(K, std=0.1))
    layer.quantize_weight()
    layer.zero_grad()
    batches = []
    for _ in range(2):
        x, r, dy, dres = normal(T, K), normal(T, K, std=2.0), normal(T, N, std=1e-3), normal(T, K, std=1e-3)
        layer.forward(x, r)
        layer.backward(dy, dres)
        batches.append({k: to_np(v).astype(np.float64) for k, v in dict(
            x=x, r=r, dres=dres, h=layer.h, rstd=layer.rstd, y=layer.y, dxn=layer.dxn, dh=layer.dh,
            x8=wide(layer.x8[0], layer.x8[1], "e4m3"), x8t=wide(layer.x8[2], layer.x8[3], "e4m3"),
            g8=wide(layer.g8[0], layer.g8[1], "e5m2"), g8t=wide(layer.g8[2], layer.g8[3], "e5m2")).items()})
    s = dict(batches=batches, gamma=to_np(layer.gamma).astype(np.float64),
             w8=to_np(wide(layer.w8[0], layer.w8[1], "e4m3")), w8t=to_np(wide(layer.w8[2], layer.w8[3], "e4m3")),
             dweight=to_np(layer.dweight).astype(np.float64), dgamma=to_np(layer.dgamma).astype(np.float64))
    s["norm"] = layer.clip().item()
    s["clipped"] = [to_np(t).astype(np.float64) for t in (layer.dweight, layer.dgamma)]
    return s


def wide(codes, scales, fmt):
    """MXFP8 values: a code times its block's power of two."""
    import torch

    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)
    return codes.view(kind).double() * step


def product(a, b, half):
    """(a b^T, how far the library's may be)."""
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    loss = 2 * U * a.shape[1] * mag
    return ref, loss + half * (np.abs(ref) + loss)


def test_products(step):
    for b in step["batches"]:
        ref, most = product(b["x8"], step["w8"], 2.0 ** -8)
        assert (np.abs(b["y"] - ref) <= most).all()
        ref, most = product(b["g8"], step["w8t"], 2.0 ** -8)
        assert (np.abs(b["dxn"] - ref) <= most).all()


def test_norm_output_is_what_was_quantized(step):
    """An E4M3 code is off by at most 2^-4 of the value, or by half of the smallest
    step, 2^-10 of the block's scale, which is at most its maximum / 224."""
    for b in step["batches"]:
        y = oracle.norm.normed(b["h"], b["rstd"], step["gamma"])
        blocks = np.abs(y).reshape(T, K // 32, 32).max(axis=2).repeat(32, axis=1)
        assert (np.abs(b["x8"] - y) <= 2.0 ** -4 * np.abs(y) * 1.001 + blocks * 2.0 ** -10 / 224).all()


def test_norm_gradient(step):
    """dh itself, and the share of it that is not dres."""
    for b in step["batches"]:
        ref, _ = oracle.norm.norm_bwd(b["dxn"], b["h"], b["rstd"], step["gamma"], b["dres"])
        most = oracle.norm.norm_bwd_bound(b["dxn"], b["h"], b["rstd"], step["gamma"], b["dres"], longest(K), 2.0 ** -8)
        assert (np.abs(b["dh"] - ref) <= most).all()
        share = ref - b["dres"]
        off = (b["dh"] - b["dres"]) - share
        # the bf16 rounding of dh: uniform within half a step at most, so a third of its square
        rounding = 2.0 ** -8 * np.sqrt((ref ** 2).mean() / 3)
        assert np.sqrt((off ** 2).mean()) <= rounding * 1.01


def test_main_gradients(step):
    ref, most, dref, dmag = 0, 0, 0, 0
    for b in step["batches"]:
        r, m = product(b["g8t"], b["x8t"], 0.0)
        ref, most = ref + r, most + m
        term = b["dxn"] * b["h"] * b["rstd"][:, None]
        dref, dmag = dref + term.sum(axis=0), dmag + np.abs(term).sum(axis=0)
    most = most + 4 * U * np.abs(ref)
    assert (np.abs(step["dweight"] - ref) <= most).all()
    # a call's own roundings, and the rounding of the accumulator after the first call
    assert (np.abs(step["dgamma"] - dref) <= bound(T, K, dmag, dref) + U * dmag).all()


def test_norm_and_clipping(step):
    total = sum((step[k] ** 2).sum() for k in ("dweight", "dgamma"))
    assert abs(step["norm"] / np.sqrt(total) - 1) <= 2 * U
    k = min(1.0, 0.25 / (np.sqrt(total) + 1e-6))
    assert k < 0.9, "the step has nothing to clip"
    for got, before in zip(step["clipped"], (step["dweight"], step["dgamma"])):
        assert (np.abs(got - before * k) <= 5 * U * np.abs(before * k)).all()
