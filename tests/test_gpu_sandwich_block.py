"""Joining norms, the router's gradient and orthogonal updates together, as
examples/sandwich_block.py uses them, and the runner's methods around them."""

import importlib.util
import os

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sandwich_block", os.path.join(ROOT, "examples", "sandwich_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_runs(example):
    losses, balance = example.main(T=128, H=256, I=160, E=8, k=2, steps=3)
    assert all(0 < v < float("inf") for v in losses + balance)


def test_gradients_against_differentiation_in_64_bits(example):
    """Of a loss on the output with the routers' losses, at the routing that the blocks
    took.  bf16 rounds n, y, h, dy, dn and d_h on the way through a block (u = 2^-8
    each, at most 0.6 u in the 2-norm), two blocks in a row: 12 roundings forward and
    backward, each carried through products that keep its relative size: 12 * 0.6 u =
    2.9e-2 if all pointed the same way."""
    T, H, I, E, k = 48, 64, 40, 4, 2
    m = example.Model(T, H, I, E, k, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d_out = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    balance, z = 0.5, 0.1
    m.forward(x)
    dx = m.backward(d_out, balance, z)

    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    xs = leaf(x)
    params = [{n: leaf(getattr(b, n)) for n in ("router", "gate_weight", "w_gate_up", "w_down", "norm_weight", "post_weight")}
              for b in m.blocks]
    norm = lambda v, w: v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    h, loss = xs, 0.0
    for b, p in zip(m.blocks, params):
        n = norm(h, p["norm_weight"])
        logits, idx = n @ p["router"], b.idx.long()
        w = torch.softmax(logits.gather(1, idx), -1)
        y = torch.zeros_like(h)
        for j in range(k):
            hid = torch.einsum("th,thi->ti", n, p["w_gate_up"][idx[:, j]])
            y = y + w[:, j:j + 1] * torch.einsum("ti,tih->th", torch.nn.functional.silu(hid[:, :I]) * hid[:, I:],
                                                 p["w_down"][idx[:, j]])
        f = torch.bincount(idx.flatten(), minlength=E).double() * E / (T * k)
        loss = loss + balance * (torch.softmax(logits, -1).mean(0) * f).sum() + z * torch.logsumexp(logits, -1).square().mean()
        h = h + torch.sigmoid(n @ p["gate_weight"])[:, None] * norm(y, p["post_weight"])
    loss = loss + (h * d_out.double()).sum()
    names = [(i, n) for i, p in enumerate(params) for n in p]
    ref = torch.autograd.grad(loss, [xs] + [params[i][n] for i, n in names])

    def close(what, got, want):
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 2.9e-2, (what, err)

    close("x", dx, ref[0])
    for (i, n), want in zip(names, ref[1:]):
        b = m.blocks[i]
        got = {"w_gate_up": b.layer.dw_gate_up, "w_down": b.layer.dw_down}.get(n)
        close((i, n), getattr(b, "d_" + n) if got is None else got, want)


def test_runner_orthogonalize(example):
    E, H, I = 3, 144, 200
    r = LayerRunner(8, H, I, E, 2, moe.MOE_ACT_SWIGLU)
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (r.dw_gate_up, r.dw_down):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    ug, ud = r.orthogonalize(scale=0.5)
    ws = moe.orthogonalize_workspace(r.dw_down)
    for got, src in ((ug[:, :, :I], r.dw_gate_up[:, :, :I]), (ug[:, :, I:], r.dw_gate_up[:, :, I:]), (ud, r.dw_down)):
        want = torch.empty(src.shape, dtype=torch.bfloat16, device="cuda")
        moe.orthogonalize(src.contiguous(), want, ws, scale=0.5)
        assert torch.equal(got, want)
    # given momenta, on another stream, again in the same buffers
    mg, md = r.dw_gate_up.to(torch.bfloat16), 2 * r.dw_down
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ug2, ud2 = r.orthogonalize(mg, md, stream=s)
    torch.cuda.synchronize()
    assert ug2 is ug and ud2 is ud
    want = torch.empty_like(ud)
    moe.orthogonalize(md, want, ws)
    torch.cuda.synchronize()
    assert torch.equal(ud2, want)
    r.check()
    with pytest.raises(ValueError):
        r.orthogonalize(md, mg)
    with pytest.raises(ValueError):
        LayerRunner(8, H, I, E, 2, moe.MOE_ACT_SWIGLU, gate_up_layout=1).orthogonalize()


def test_runner_route_bwd():
    T, H, I, E, k = 40, 64, 32, 8, 2
    r = LayerRunner(T, H, I, E, k, moe.MOE_ACT_SWIGLU)
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn((T, E), generator=g, device="cuda")
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    r.route(logits, idx, w)
    r.d_topk_w.copy_(torch.randn((T, k), generator=g, device="cuda"))
    d, losses = r.route_bwd(logits, idx, w, balance=0.1, z=0.01)
    want, wl = torch.empty_like(d), torch.empty_like(losses)
    counts = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
    moe.route_bwd(r.shape, logits, want, moe.route_bwd_workspace(r.shape), idx, w, r.d_topk_w, counts, 0.1, 0.01, wl)
    assert torch.equal(d, want) and torch.equal(losses, wl)
    other = torch.randn((T, k), generator=g, device="cuda")
    d2, _ = r.route_bwd(logits, idx, w, other)
    moe.route_bwd(r.shape, logits, want, moe.route_bwd_workspace(r.shape), idx, w, other)
    # (with the losses wanted the softmax runs too, its factors 0)
    assert (d2 - want).abs().max() <= 2.0 ** -24 * want.abs().max()
    r.check()


def test_a_step_in_a_graph(example):
    """Forward, backward and updates of a block, captured after a run in the eager
    mode whose results are still held, give the same bits when replayed."""
    T, H, I, E, k = 64, 64, 136, 4, 2
    m = example.Model(T, H, I, E, k, 1)
    b = m.blocks[0]
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d_out = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))

    def go():
        m.forward(x)
        m.backward(d_out, 0.1, 0.01)
        b.layer.orthogonalize()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    out = (b.h, m.dx, b.layer.u_gate_up, b.layer.u_down, b.layer.dw_gate_up, b.layer.d_logits, b.layer.losses, b.d_post_weight)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for t in out:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for t, v in zip(out, want):
        assert torch.equal(t, v)
    b.layer.check()
