"""Global gradient norm and clipping against the definition in 64 bits.

The norm: squares are rounded (u32 each), up to 8192 / 256 of them are added in
fp32 by a thread, the rest in 64 bits; the root halves the relative error:
(32 + 4) / 2 half-steps bound it.  The factor adds its own rounding, the
scaled gradient the product's and the type's."""

import math

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
NORM_REL = 18 * U32


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tensors(sizes, dts, std=0.01, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(dts[i % len(dts)]) for i, n in enumerate(sizes)]


def run(grads, max_norm, out=None):
    t = moe.grad_table(grads, out)
    norm = torch.empty(2, device="cuda")
    ws = moe.grad_clip_workspace(t)
    moe.grad_clip(t, max_norm, norm, ws)
    again = torch.empty(2, device="cuda")
    if out is not None and out is not False:      # the workspace is ready for the next call
        moe.grad_clip(t, max_norm, again, ws)
        assert torch.equal(norm.view(torch.int32), again.view(torch.int32))
    return norm.cpu()


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check(sizes, dts, factor, seed=0, in_place=False):
    host = tensors(sizes, dts, seed=seed)
    dev = [t.cuda() for t in host]
    nx = exact_norm(host)
    out = None if in_place else [torch.full_like(t, 9.0) for t in dev]
    norm = run(dev, nx * factor, out)
    assert abs(norm[0].item() - nx) <= (NORM_REL + U32) * nx
    cx = min(1.0, float(torch.tensor(nx * factor, dtype=torch.float32)) / (nx + 1e-6)) if nx else 1.0
    assert abs(norm[1].item() - cx) <= (NORM_REL + 2 * U32) * cx
    for t, o in zip(host, dev if in_place else out):
        ref = t.double() * cx
        bound = (half_step(t.dtype) + NORM_REL + 3 * U32) * ref.abs()
        if t.dtype is torch.bfloat16:   # a bf16 tie may fall on either side of the fp32 product
            bound = bound * (1 + 1e-6)
        assert torch.all((o.cpu().double() - ref).abs() <= bound)


@pytest.mark.parametrize("sizes", [[1], [7], [8192], [8193], [5, 0, 3, 100000], [1 << 20, 17, 4097],
                                   [12345] * 40])
@pytest.mark.parametrize("dts", [[torch.float32], [torch.bfloat16], [torch.float32, torch.bfloat16]])
def test_clip(sizes, dts):
    check(sizes, dts, 0.3)
    check(sizes, dts, 3.0)
    check(sizes, dts, 0.3, in_place=True)


def test_more_tensors_than_one_launch_takes():
    check([100 + 7 * i for i in range(300)], [torch.float32, torch.bfloat16], 0.5)


def test_unaligned_slices():
    base = tensors([10001], [torch.float32])[0]
    flat = base.cuda()
    views, host = [], []
    for a, b in [(1, 1000), (1003, 5000), (5001, 10001)]:
        views.append(flat[a:b])
        host.append(base[a:b])
    nx = exact_norm(host)
    outs = [torch.empty(20003, device="cuda")[3:3 + v.numel()] for v in views]
    norm = run(views, 0.5 * nx, outs)
    assert abs(norm[0].item() - nx) <= (NORM_REL + U32) * nx
    for h, o in zip(host, outs):
        ref = h.double() * (0.5 * nx / (nx + 1e-6))
        assert torch.all((o.cpu().double() - ref).abs() <= (NORM_REL + 4 * U32) * ref.abs())


@pytest.mark.parametrize("std", [1e-38, 1e-25, 1e-13, 1e-7, 1e10, 1e19, 1e30])
def test_range(std):
    host = tensors([3000, 17], [torch.float32], std)
    nx = exact_norm(host)
    norm = run([t.cuda() for t in host], float("inf"), False)
    # below 2^-126 the values themselves carry fewer bits; their squares are scaled up
    assert abs(norm[0].item() - nx) <= (NORM_REL + U32) * nx + 2.0 ** -149
    assert norm[1].item() == 1.0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_leaves_the_gradients(bad):
    host = tensors([100, 20000], [torch.float32])
    host[1][15000] = bad
    dev = [t.cuda() for t in host]
    out = [torch.zeros_like(t) for t in dev]
    norm = run(dev, 1e-3, out)
    assert norm[0].item() == float("inf") if math.isinf(bad) else math.isnan(norm[0].item())
    assert norm[1].item() == 1.0
    for t, o in zip(host, out):
        assert torch.equal(o.cpu().view(torch.int32), t.view(torch.int32))


def test_empty_and_zero():
    assert run([], 1.0, []).tolist() == [0.0, 1.0]
    z = torch.zeros(100, device="cuda")
    assert run([z, torch.empty(0, device="cuda")], 1.0).tolist() == [0.0, 1.0]
    g = torch.ones(100, device="cuda")
    n = run([g], 0.0, [z])
    assert n[0].item() == 10.0 and n[1].item() == 0.0 and torch.all(z == 0)


def test_graph_and_repeatable():
    dev = [t.cuda() for t in tensors([100000, 333, 5000], [torch.float32])]
    out = [torch.empty_like(t) for t in dev]
    t = moe.grad_table(dev, out)
    norm, ws = torch.empty(2, device="cuda"), moe.grad_clip_workspace(t)
    moe.grad_clip(t, 0.1, norm, ws)
    first = [norm.clone()] + [o.clone() for o in out]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.grad_clip(t, 0.1, norm, ws)
    for _ in range(3):
        norm.zero_()
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, [norm] + out))
