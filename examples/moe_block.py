"""A pre-norm residual block around the expert layer, trained for a few steps and
then served token by token on 4-bit weights.

    total = x + residual
    n     = rms_norm(total) * norm_weight
    route = top-k of n @ router
    out   = total + experts(n)

Training uses rms_norm_fwd / rms_norm_bwd around LayerRunner's forward and
backward and clips all gradients by their global norm (LayerRunner.clip_grads);
serving quantises the expert weights once (LayerRunner.quantize), takes the norm
in 8 bits and runs the few-token layer (LayerRunner.few).  The router's product and
the update are plain torch.

    python examples/moe_block.py
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner


class Block:
    def __init__(self, T, H, I, E, k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.T, self.H, self.E, self.k = T, H, E, k
        self.norm_weight = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.router = normal((H, E), H ** -0.5)
        self.w_gate_up = normal((E, H, 2 * I), H ** -0.5).to(torch.bfloat16)
        self.w_down = normal((E, I, H), I ** -0.5).to(torch.bfloat16)
        self.layer = LayerRunner(T, H, I, E, k, moe.MOE_ACT_SWIGLU)
        self.n, self.total = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.rstd = torch.empty(T, device="cuda")
        self.idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
        self.w = torch.empty((T, k), device="cuda")
        self.d_norm_weight = torch.empty(H, device="cuda")
        self.dx = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        self.ws_norm = moe.rms_norm_workspace(T, H)

    def forward(self, x, residual):
        moe.rms_norm_fwd(x, self.norm_weight, self.n, residual=residual, total=self.total, rstd=self.rstd)
        self.layer.route(self.n.float() @ self.router, self.idx, self.w)
        y = self.layer.forward(self.n, self.idx, self.w, self.w_gate_up, self.w_down)
        return self.total + y

    def backward(self, d_out):
        """Gradients of the parameters (in self.layer and here) and of x."""
        dn, dw, _, _ = self.layer.backward(d_out, self.n, self.idx, self.w, self.w_gate_up, self.w_down)
        # softmax over the chosen logits
        d_chosen = self.w * (dw - (self.w * dw).sum(-1, keepdim=True))
        d_logits = torch.zeros((self.T, self.E), device="cuda").scatter_(1, self.idx.long(), d_chosen)
        self.d_router = self.n.float().t() @ d_logits
        dn = (dn.float() + d_logits @ self.router.t()).to(torch.bfloat16)
        moe.rms_norm_bwd(dn, self.total, self.rstd, self.norm_weight, self.dx, self.d_norm_weight,
                         d_total=d_out, ws=self.ws_norm)
        return self.dx

    def step(self, x, residual, target, lr, max_norm):
        """One step on the mean squared error; (loss, gradient norm)."""
        out = self.forward(x, residual)
        diff = out.float() - target
        self.backward((2 / diff.numel() * diff).to(torch.bfloat16))
        norm = self.layer.clip_grads(max_norm, extra=[self.d_router, self.d_norm_weight])
        for p, g in ((self.w_gate_up, self.layer.dw_gate_up), (self.w_down, self.layer.dw_down),
                     (self.router, self.d_router), (self.norm_weight, self.d_norm_weight)):
            p.copy_(p.float() - lr * g)
        return diff.square().mean(), norm[0].clone()

    def server(self, tokens=1):
        """A function (x, residual) -> out for `tokens` tokens on the present
        weights in 4 bits."""
        T, H = tokens, self.H
        layer = LayerRunner(T, H, self.w_down.shape[1], self.E, self.k, moe.MOE_ACT_SWIGLU,
                            training=False, backward=False)
        layer.quantize(self.w_gate_up, self.w_down)
        n8, scale = (torch.empty((T, w), dtype=torch.uint8, device="cuda") for w in (H, H // 32))
        total = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        idx = torch.empty((T, self.k), dtype=torch.int32, device="cuda")
        w = torch.empty((T, self.k), device="cuda")

        def serve(x, residual):
            moe.rms_norm_fwd(x, self.norm_weight, n8, residual=residual, total=total, y_scale=scale)
            n = n8.view(torch.float8_e4m3fn).float() * torch.exp2(scale.float() - 127).repeat_interleave(32, 1)
            moe.route(layer.shape, n @ self.router, idx, w)
            return total + layer.few(n8, idx, w, x_scale=scale)

        return serve


def main(T=256, H=512, I=256, E=16, k=4, steps=30, lr=5.0, max_norm=0.3):
    """(losses, gradient norms, relative difference of the served outputs)."""
    block = Block(T, H, I, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    target = (x.float() + residual.float()).roll(1, dims=1)
    losses, norms = [], []
    for _ in range(steps):
        loss, norm = block.step(x, residual, target, lr, max_norm)
        losses.append(loss)
        norms.append(norm)
    out = block.forward(x, residual)
    serve = block.server(1)
    served = torch.cat([serve(x[t:t + 1], residual[t:t + 1]) for t in range(32)])
    block.layer.check()
    y, ys = (out - block.total)[:32].float(), (served - block.total[:32]).float()
    return [float(v) for v in losses], [float(v) for v in norms], float((ys - y).norm() / y.norm())


if __name__ == "__main__":
    losses, norms, rel = main()
    print("loss %.4f -> %.4f, gradient norm %.3g -> %.3g" % (losses[0], losses[-1], norms[0], norms[-1]))
    print("experts' output on 4-bit weights and 8-bit tokens: relative difference %.3f" % rel)
