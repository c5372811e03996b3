"""Workspaces that other calls have used: a call's result does not depend on what
its workspace holds (but for the error word, which the first zero-fill clears)."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from test_gpu_few import CLAMPED, SWIGLU, make, run
from test_gpu_grad_clip import tensors

pytestmark = pytest.mark.gpu

KINDS = [("bf16", False), ("bf16", True), ("fp32", False), ("mx", False), ("mx", True)]


def used(n):
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    return ws


def shape_of(c):
    return moe.Shape(c["T"], c["H"], c["I"], c["E"], c["k"], c["act"],
                     moe.MOE_FP32 if c["weights"] == "fp32" else moe.MOE_BF16, 7.0, 1.702, 0, 0)


@pytest.mark.parametrize("weights,x8", KINDS)
@pytest.mark.parametrize("T,H,I", [(1, 1088, 544), (5, 4160, 96), (20, 288, 320)])
def test_few_on_a_used_workspace(weights, x8, T, H, I):
    c = make(T, H, I, 6, 3, SWIGLU, weights, x8=x8, bias=True)
    right, _ = run(c)
    y, ws = run(c, ws=used(moe.moe_few_workspace_size(shape_of(c))))
    moe.check_device_error(ws)
    assert torch.equal(y, right)


@pytest.mark.parametrize("weights,x8", KINDS)
def test_few_of_two_shapes_in_turn(weights, x8):
    small = make(6, 64, 1056, 4, 2, SWIGLU, weights, x8=x8)
    large = make(3, 8224, 64, 4, 2, CLAMPED, weights, x8=x8, seed=1)
    right = [run(c)[0] for c in (small, large)]
    ws = torch.zeros(max(moe.moe_few_workspace_size(shape_of(c)) for c in (small, large)),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c, r in zip((small, large), right):
            assert torch.equal(run(c, ws=ws)[0], r)
    moe.check_device_error(ws)


def test_prompt_and_decode_on_one_workspace():
    few = make(9, 264, 136, 8, 2, SWIGLU)
    many = make(300, 264, 136, 8, 2, SWIGLU, seed=1)
    s_few, s_many = shape_of(few), shape_of(many)
    ws = torch.zeros(max(moe.moe_few_workspace_size(s_few), moe.moe_workspace_size(s_many, 1)),
                     dtype=torch.uint8, device="cuda")
    right, _ = run(few)
    d = [many[n].cuda() for n in ("x", "idx", "w", "w_gate_up", "w_down")]
    first = None
    for _ in range(2):
        y = torch.full((300, 264), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ffn_fwd(s_many, *d, y, ws)
        first = y if first is None else first
        assert torch.equal(y, first)
        assert torch.equal(run(few, ws=ws)[0], right)
    moe.check_device_error(ws)


@pytest.mark.parametrize("sizes", [[5], [1000, 3, 70000], [333] * 250, [4 << 20]])
@pytest.mark.parametrize("scaled", [True, False])
def test_grad_clip_on_a_used_workspace(sizes, scaled):
    dev = [t.cuda() for t in tensors(sizes, [torch.float32, torch.bfloat16])]
    out = []
    for fill in (False, True):
        dst = [torch.full_like(t, 9.0) for t in dev]
        t = moe.grad_table(dev, dst if scaled else False)
        ws = moe.grad_clip_workspace(t)
        if fill:
            ws = used(ws.numel())
        norm = torch.full((2,), -1.0, device="cuda")
        moe.grad_clip(t, 0.01, norm, ws)
        out.append([norm] + dst)
    assert out[0][0][0] > 0
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_clip_and_few_on_one_workspace():
    c = make(4, 320, 96, 6, 2, SWIGLU, "mx")
    right, _ = run(c)
    dev = [t.cuda() for t in tensors([5000, 70000], [torch.float32])]
    t = moe.grad_table(dev, False)
    ws = torch.zeros(max(moe.moe_few_workspace_size(shape_of(c)), moe.grad_clip_workspace(t).numel()),
                     dtype=torch.uint8, device="cuda")
    norm, first = torch.empty(2, device="cuda"), None
    for _ in range(2):
        moe.grad_clip(t, 1.0, norm, ws)
        first = norm.clone() if first is None else first
        assert torch.equal(norm, first)
        assert torch.equal(run(c, ws=ws)[0], right)


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_FP32])
@pytest.mark.parametrize("recompute", [False, True])
def test_the_layer_on_used_workspaces(dtype, recompute):
    from dispatch_gemm_combine_gb300.runner import LayerRunner
    c = make(70, 264, 136, 8, 2, SWIGLU, "fp32" if dtype == moe.MOE_FP32 else "bf16")
    a = [c[n].cuda() for n in ("x", "idx", "w", "w_gate_up", "w_down")]
    out = []
    for fill in (False, True):
        r = LayerRunner(70, 264, 136, 8, 2, SWIGLU, dtype)
        r.ws_bwd_recompute = moe.workspace(r.shape, 3)
        if fill:
            for ws in (r.ws_plan, r.ws_fwd, r.ws_bwd, r.ws_bwd_recompute):
                ws[256:] = 0xA5
        r.plan(a[1])
        y = r.forward(*a).clone()
        out.append((y,) + tuple(t.clone() for t in r.backward(a[0], *a, recompute=recompute)))
        r.check()
    assert all(torch.equal(p, q) for p, q in zip(*out))
