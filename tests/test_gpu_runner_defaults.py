"""What LayerRunner's methods take where no gradient is given: zeros before the first
backward, whatever the memory held, and never the gradient of an earlier step."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner

pytestmark = pytest.mark.gpu

T, H, I, E, K = 40, 64, 32, 8, 2


@pytest.fixture(autouse=True)
def memory_that_held_nan(monkeypatch):
    empty = torch.empty

    def held_nan(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(float("nan")) if t.is_floating_point() else t

    monkeypatch.setattr(torch, "empty", held_nan)


def runner(**kw):
    return LayerRunner(T, H, I, E, K, moe.MOE_ACT_SWIGLU, **kw)


def inputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf16 = lambda *s: normal(*s).to(torch.bfloat16)  # noqa: E731
    logits = normal(T, E)
    idx, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    return logits, idx, w, bf16(T, H), bf16(T, H), 0.1 * bf16(E, H, 2 * I), 0.1 * bf16(E, I, H)


def test_before_the_first_backward():
    logits, idx, w = inputs()[:3]
    r, losses_only = runner(), runner(backward=False)
    for a in (r, losses_only):
        a.route(logits, idx, w)
    d, losses = r.route_bwd(logits, idx, w, balance=0.1, z=0.01)
    want, want_losses = losses_only.route_bwd(logits, idx, w, balance=0.1, z=0.01)
    assert torch.isfinite(d).all() and d.any()
    assert torch.equal(d, want) and torch.equal(losses, want_losses)
    assert not any(u.any() for u in r.orthogonalize())
    assert r.clip_grads(1.0)[0] == 0


def test_router_gradient_is_never_of_an_earlier_step():
    logits, idx, w, x, dy, wgu, wd = inputs()
    r = runner()

    def forward(**kw):
        r.route(logits, idx, w)
        r.forward(x, idx, w, wgu, wd, **kw)

    forward()
    with pytest.raises(ValueError):
        r.route_bwd(logits, idx, w)
    r.backward(dy, x, idx, w, wgu, wd)
    right = r.route_bwd(logits, idx, w)[0].clone()
    assert right.any()
    for kw in ({}, dict(inference=True)):
        forward(**kw)
        with pytest.raises(ValueError):
            r.route_bwd(logits, idx, w, balance=0.1)
        # ... but the one that is meant may be given
        assert torch.equal(r.route_bwd(logits, idx, w, r.d_topk_w)[0], right)
        forward()
        r.backward(dy, x, idx, w, wgu, wd)
        assert torch.equal(r.route_bwd(logits, idx, w)[0], right)
    r.check()
