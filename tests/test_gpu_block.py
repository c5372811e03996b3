"""The operators together, as examples/moe_block.py uses them, and the runner's
methods around them."""

import importlib.util
import os

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_and_serving(example):
    losses, norms, rel = example.main(T=128, H=256, I=128, E=8, k=2, steps=20)
    assert losses[-1] < 0.7 * losses[0]
    assert all(0 < n < float("inf") for n in norms)
    # 4-bit weights are off by up to 1/4 of a value at 1 (half a step of 0.5 over 1 .. 2 is
    # 1/4 .. 1/8, with a uniform spread about 0.1), through two products
    assert rel < 0.3


def test_gradient_of_the_block_against_differences(example):
    """<dx, d> of the bf16 block against central differences of the same block in
    64 bits at the routing that it took.  bf16 rounds n, y and dn (u = 2^-8 each,
    three times in a row along the path): 4 u of the terms' magnitudes."""
    T, H, I, E, k = 16, 64, 32, 4, 2
    b = example.Block(T, H, I, E, k)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r, d_out, d = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    b.forward(x, r)
    dx = b.backward(d_out).double()
    idx = b.idx.long()
    wgu, wd, router, nw = (t.double() for t in (b.w_gate_up, b.w_down, b.router, b.norm_weight))

    def f(xv):
        total = xv + r.double()
        n = total / torch.sqrt(total.square().mean(-1, keepdim=True) + 1e-6) * nw
        w = torch.softmax((n @ router).gather(1, idx), -1)
        y = torch.zeros_like(total)
        for j in range(k):
            h = torch.einsum("th,thi->ti", n, wgu[idx[:, j]])
            a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            y = y + w[:, j:j + 1] * torch.einsum("ti,tih->th", a, wd[idx[:, j]])
        return (d_out.double() * (total + y)).sum()

    e = 1e-5
    num = (f(x.double() + e * d.double()) - f(x.double() - e * d.double())) / (2 * e)
    assert abs((dx * d.double()).sum() - num) <= 4 * 2.0 ** -8 * (dx * d.double()).abs().sum()


def test_clip_grads_scales_in_place():
    from dispatch_gemm_combine_gb300.runner import LayerRunner
    r = LayerRunner(8, 64, 32, 4, 2, moe.MOE_ACT_SWIGLU)
    g = torch.Generator(device="cuda").manual_seed(2)
    r.dw_gate_up.normal_(generator=g)
    r.dw_down.normal_(generator=g)
    extra = torch.randn(100, generator=g, device="cuda").to(torch.bfloat16)
    before = [t.double().clone() for t in (r.dw_gate_up, r.dw_down, extra)]
    nx = torch.sqrt(sum(t.square().sum() for t in before))
    out = r.clip_grads(1.5, extra=[extra])
    assert abs(out[0].double() - nx) <= 1e-6 * nx
    for t, b, u in zip((r.dw_gate_up, r.dw_down, extra), before, (2.0 ** -24, 2.0 ** -24, 2.0 ** -8)):
        ref = b * 1.5 / (nx + 1e-6)
        assert torch.all((t.double() - ref).abs() <= (u + 2e-6) * ref.abs())
    out = r.clip_grads(10.0)      # fewer tensors, nothing to clip
    assert out[1].item() == 1.0


def test_few_needs_weights():
    from dispatch_gemm_combine_gb300.runner import LayerRunner
    r = LayerRunner(1, 64, 32, 4, 2, moe.MOE_ACT_SWIGLU, training=False, backward=False)
    x = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    idx, w = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros((1, 2), device="cuda")
    with pytest.raises(ValueError):
        r.few(x, idx, w)
