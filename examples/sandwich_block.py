"""Blocks with a norm before and after the experts, trained with the router's losses
and orthogonal weight updates.

    n_0 = rms_norm(h_0) * norm_weight_0
    for each block:
      route   = top-k of n @ router
      y       = experts(n)
      h      <- h + sigmoid(n @ gate_weight) * rms_norm(y) * post_weight     (per token)
      n       = rms_norm(h) * norm_weight of the next block

join_norm_fwd / join_norm_bwd take the two norms, the gate and the residual's addition
in one call; LayerRunner.route_bwd gives the router's gradient with the load-balancing
and z-losses; the gradients are clipped by their global norm (LayerRunner.clip_grads)
and the expert weights follow the orthogonalised momenta of theirs
(LayerRunner.orthogonalize).  The other products and updates are plain torch.

    python examples/sandwich_block.py
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner

BF16 = torch.bfloat16


class Block:
    def __init__(self, T, H, I, E, k, normal):
        self.router, self.gate_weight = normal((H, E), H ** -0.5), normal((H,), H ** -0.5)
        self.w_gate_up = normal((E, H, 2 * I), H ** -0.5).to(BF16)
        self.w_down = normal((E, I, H), I ** -0.5).to(BF16)
        self.norm_weight, self.post_weight = (torch.ones(H, dtype=BF16, device="cuda") for _ in range(2))
        self.layer = LayerRunner(T, H, I, E, k, moe.MOE_ACT_SWIGLU)
        self.n, self.y, self.h, self.dy = (torch.empty((T, H), dtype=BF16, device="cuda") for _ in range(4))
        self.rstd, self.rstd_post, self.gate, self.d_gate = (torch.empty(T, device="cuda") for _ in range(4))
        self.idx, self.w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
        self.d_norm_weight, self.d_post_weight = (torch.empty(H, device="cuda") for _ in range(2))
        self.momenta = None

    def experts(self):
        """Routing, gates and the experts' output y of the block's input n."""
        n = self.n.float()
        self.logits = n @ self.router
        torch.sigmoid(n @ self.gate_weight, out=self.gate)
        self.layer.route(self.logits, self.idx, self.w)
        self.y.copy_(self.layer.forward(self.n, self.idx, self.w, self.w_gate_up, self.w_down))

    def experts_bwd(self, balance, z):
        """The gradient of n, from dy and d_gate; those of the parameters stay here."""
        dn = self.layer.backward(self.dy, self.n, self.idx, self.w, self.w_gate_up, self.w_down)[0]
        d_logits, self.losses = self.layer.route_bwd(self.logits, self.idx, self.w, balance=balance, z=z)
        d_pre = self.d_gate * self.gate * (1 - self.gate)
        n = self.n.float()
        self.d_router, self.d_gate_weight = n.t() @ d_logits, n.t() @ d_pre
        return (dn.float() + d_logits @ self.router.t() + d_pre[:, None] * self.gate_weight).to(BF16)


class Model:
    def __init__(self, T, H, I, E, k, blocks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.blocks = [Block(T, H, I, E, k, normal) for _ in range(blocks)]
        self.ws, self.ws_norm = moe.join_norm_workspace(T, H), moe.rms_norm_workspace(T, H)
        self.d_h, self.dx = (torch.empty((T, H), dtype=BF16, device="cuda") for _ in range(2))

    def forward(self, h):
        first = self.blocks[0]
        self.h0 = h
        moe.rms_norm_fwd(h, first.norm_weight, first.n, rstd=first.rstd)
        for b, after in zip(self.blocks, self.blocks[1:] + [None]):
            b.experts()
            moe.join_norm_fwd(b.y, h, b.h, post_weight=b.post_weight, gate=b.gate, rstd_post=b.rstd_post,
                              weight=after.norm_weight if after else None, n=after.n if after else None,
                              rstd=after.rstd if after else None)
            h = b.h
        return h

    def backward(self, d_out, balance, z):
        """Gradients of the parameters (in the blocks) and of the input."""
        d_total, dn = d_out, None
        for b, after in reversed(list(zip(self.blocks, self.blocks[1:] + [None]))):
            moe.join_norm_bwd(b.y, b.dy, self.d_h, d_total=d_total, dn=dn, total=b.h if after else None,
                              weight=after.norm_weight if after else None, rstd=after.rstd if after else None,
                              post_weight=b.post_weight, rstd_post=b.rstd_post, gate=b.gate, d_gate=b.d_gate,
                              d_post_weight=b.d_post_weight, d_weight=after.d_norm_weight if after else None, ws=self.ws)
            dn, d_total = b.experts_bwd(balance, z), self.d_h
        first = self.blocks[0]
        moe.rms_norm_bwd(dn, self.h0, first.rstd, first.norm_weight, self.dx, first.d_norm_weight, d_total=d_total,
                         ws=self.ws_norm)
        return self.dx

    def step(self, x, target, lr, beta=0.9, max_norm=1.0, balance=0.01, z=0.001):
        """One step on the mean squared error: (loss, balance losses of the blocks)."""
        diff = self.forward(x).float() - target
        self.backward((2 / diff.numel() * diff).to(BF16), balance, z)
        for b in self.blocks:
            b.layer.clip_grads(max_norm, extra=[b.d_router, b.d_gate_weight, b.d_norm_weight, b.d_post_weight])
            grads = (b.layer.dw_gate_up, b.layer.dw_down)
            if b.momenta is None:
                b.momenta = [torch.zeros_like(g) for g in grads]
            torch._foreach_lerp_(b.momenta, grads, 1 - beta)
            # updates of the same size an entry whatever the matrix: sqrt(max(M, N)) 0.2
            scale = 0.2 * max(b.w_down.shape[1:]) ** 0.5
            for p, u in zip((b.w_gate_up, b.w_down), b.layer.orthogonalize(*b.momenta, scale=scale)):
                p.add_(u, alpha=-lr)
            for p, g in ((b.router, b.d_router), (b.gate_weight, b.d_gate_weight), (b.norm_weight, b.d_norm_weight),
                         (b.post_weight, b.d_post_weight)):
                p.copy_(p.float() - lr * g)
        return diff.square().mean(), torch.stack([b.losses[0] for b in self.blocks])


def main(T=256, H=512, I=320, E=16, k=4, blocks=2, steps=30, lr=0.02):
    """(losses, the balance losses of the last step)."""
    model = Model(T, H, I, E, k, blocks)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    target = x.float() + x.float().roll(1, dims=1)
    losses = []
    for _ in range(steps):
        loss, balance = model.step(x, target, lr)
        losses.append(loss)
    for b in model.blocks:
        b.layer.check()
    return [float(v) for v in losses], balance.tolist()


if __name__ == "__main__":
    losses, balance = main()
    print("loss %.4f -> %.4f, balance losses %s" % (losses[0], losses[-1], ", ".join("%.3f" % v for v in balance)))
