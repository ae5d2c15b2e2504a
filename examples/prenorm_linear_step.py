"""One training step of a pre-norm Linear in MXFP8, from the residual stream to
clipped main gradients.

    h  = x + residual                          (the new residual stream)
    Y  = Q(norm(h) gamma) Q(W)^T               fprop
    dX = Q(dY) Q(W), dW += Q(dY)^T Q(norm(h))  dgrad, wgrad into fp32
    dh = norm backward of dX + dres, dgamma += ...
    clip dW and dgamma by their global norm

Run as a program it does a few steps on random data and prints how far each
result is from the same step in fp32.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantize_scaled_gemm_amd as q  # noqa: E402

EPS = 1e-5


class PreNormLinear:
    """Buffers of a pre-norm Linear (N x K weight) for a fixed token count; the
    library allocates nothing itself, so they are made once here."""

    def __init__(self, tokens, K, N, device="cuda", max_norm=1.0):
        T = tokens
        self.max_norm = max_norm
        bf = dict(device=device, dtype=torch.bfloat16)
        u8 = dict(device=device, dtype=torch.uint8)
        self.gamma = torch.ones(K, **bf)
        self.weight = torch.empty(N, K, **bf)
        # FP8 copies: row-wise and transposed, each with its E8M0 scales
        self.w8 = [torch.empty(N, K, **u8), torch.empty(N, K // 32, **u8), torch.empty(K, N, **u8), torch.empty(K, N // 32, **u8)]
        self.x8 = [torch.empty(T, K, **u8), torch.empty(T, K // 32, **u8), torch.empty(K, T, **u8), torch.empty(K, T // 32, **u8)]
        self.g8 = [torch.empty(T, N, **u8), torch.empty(T, N // 32, **u8), torch.empty(N, T, **u8), torch.empty(N, T // 32, **u8)]
        self.h = torch.empty(T, K, **bf)
        self.rstd = torch.empty(T, device=device)
        self.y = torch.empty(T, N, **bf)
        self.dxn = torch.empty(T, K, **bf)
        self.dh = torch.empty(T, K, **bf)
        # fp32 main gradients and what clipping them needs
        self.dweight = torch.zeros(N, K, device=device)
        self.dgamma = torch.zeros(K, device=device)
        self.plan = q.qsg_grad_plan([self.dweight, self.dgamma])
        self.sumsq = torch.empty(1, device=device, dtype=torch.float64)
        self.norm = torch.empty(1, device=device)
        self.norm_ws = torch.empty(q.qsg_rmsnorm_bwd_workspace(T, K), **u8)
        self.clip_ws = torch.empty(q.GRAD_WORKSPACE_BYTES, **u8)

    def quantize_weight(self):
        a, s, at, st = self.w8
        q.qsg_quantize(self.weight, q.MXFP8, q.E4M3, a, s, at, st)

    def forward(self, x, residual):
        a, s, at, st = self.x8
        q.qsg_rmsnorm_quantize(x, self.gamma, EPS, q.MXFP8, q.E4M3, residual=residual, h=self.h, rstd=self.rstd, q=a,
                               s=s, qt=at, st=st)
        q.qsg_scaled_gemm(a, q.E4M3, q.MXFP8, s, self.w8[0], q.E4M3, q.MXFP8, self.w8[1], self.y)
        return self.y, self.h

    def backward(self, dy, dres):
        """Gradient of x and of the residual; dres is the gradient of h."""
        g, s, gt, st = self.g8
        M = q.MXFP8
        q.qsg_quantize(dy, M, q.E5M2, g, s, gt, st)
        q.qsg_scaled_gemm(g, q.E5M2, M, s, self.w8[2], q.E4M3, M, self.w8[3], self.dxn)
        q.qsg_scaled_gemm_accumulate(gt, q.E5M2, M, st, self.x8[2], q.E4M3, M, self.x8[3], self.dweight)
        q.qsg_rmsnorm_bwd(self.dxn, self.h, self.gamma, self.rstd, self.dh, dres=dres, dgamma=self.dgamma,
                          accumulate=True, workspace=self.norm_ws)
        return self.dh

    def clip(self):
        """Data-parallel ranks that hold different gradients all-reduce sumsq between the two calls."""
        q.qsg_grad_sumsq(self.plan, self.sumsq, self.clip_ws)
        q.qsg_grad_clip(self.plan, self.sumsq, self.max_norm, self.norm)
        return self.norm

    def zero_grad(self):
        self.dweight.zero_()
        self.dgamma.zero_()


def reference(layer, batches):
    """The same accumulated step in fp32: (y, dh of the last batch, dW, dgamma, norm)."""
    w, g = layer.weight.float().requires_grad_(), layer.gamma.float().requires_grad_()
    for x, r, dy, dres in batches:
        h = (x.float() + r.float()).to(x.dtype).float().requires_grad_()
        y = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * g) @ w.t()
        torch.autograd.backward([y, h], [dy.float(), dres.float()])
    norm = torch.sqrt(w.grad.double().square().sum() + g.grad.double().square().sum())
    k = min(1.0, layer.max_norm / (norm.item() + 1e-6))
    return y.detach(), h.grad, w.grad * k, g.grad * k, norm


def run(tokens=2048, K=1024, N=1536, micro_batches=2, seed=0):
    """A step of `micro_batches`; {name: relative error against fp32}."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(torch.bfloat16)

    layer = PreNormLinear(tokens, K, N, max_norm=0.25)
    layer.weight.copy_(normal(N, K, std=0.02))
    layer.gamma.copy_(1 + normal(K, std=0.1))
    layer.quantize_weight()
    layer.zero_grad()
    batches = [(normal(tokens, K), normal(tokens, K, std=2.0), normal(tokens, N, std=1e-3), normal(tokens, K, std=1e-3))
               for _ in range(micro_batches)]
    for x, r, dy, dres in batches:
        y, _ = layer.forward(x, r)
        dh = layer.backward(dy, dres)
    norm = layer.clip()
    ref = reference(layer, batches)
    got = (y.float(), dh.float(), layer.dweight, layer.dgamma, norm.double())
    names = ("y", "dh", "dweight", "dgamma", "norm")
    return {n: ((a - b).norm() / b.norm()).item() for n, a, b in zip(names, got, ref)}


if __name__ == "__main__":
    for name, err in run().items():
        print(f"{name:8s} relative error against fp32: {err:.4f}")
