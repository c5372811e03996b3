"""Waits that run out at any place of a pair's ring: each CTA of a pair waits by its own
clock, so one may have given up where the other has loaded on.  The call ends, its
error is reported (or its result is right), and the next call on the same workspace is
right.  Limits from one that no wait keeps to one that most do."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner

pytestmark = pytest.mark.gpu

LIMITS_NS = (1, 100, 300, 1000, 3000, 10000)


def with_limit(ns, call):
    before = moe.moe_set_wait_timeout_ns(ns)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_timeout_ns(before)


def ended_with_error(ws):
    try:
        moe.check_device_error(ws)
    except moe.MoeError as e:
        assert e.status == moe.MOE_ERR_TIMEOUT
        return True
    return False


@pytest.mark.parametrize("shape", [(2, 700, 900), (1, 2048, 1500), (7, 300, 1001), (3, 1300, 200)])
def test_orthogonal_updates(shape):
    g = torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    ws = moe.orthogonalize_workspace(g)
    want, out = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.orthogonalize(g, want, ws)
    moe.check_device_error(ws)
    failed = 0
    for ns in LIMITS_NS:
        for _ in range(4):
            with_limit(ns, lambda: moe.orthogonalize(g, out, ws))
            bad = ended_with_error(ws)
            failed += bad
            assert bad or torch.equal(out, want)
            moe.orthogonalize(g, out, ws)
            moe.check_device_error(ws)
            assert torch.equal(out, want)
    assert failed


@pytest.mark.parametrize("T,H,I,E,k,layout", [(2048, 512, 512, 8, 4, 0), (700, 264, 328, 5, 2, 0), (1500, 384, 256, 6, 3, 1)])
def test_the_layer(T, H, I, E, k, layout):
    """Forward and backward of the expert layer, whose products run on such pairs too."""
    g = torch.Generator(device="cuda").manual_seed(4)

    def bf16(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)

    x, dy = bf16(T, H), bf16(T, H)
    wgu, wd = bf16(E, H, 2 * I, std=H ** -0.5), bf16(E, I, H, std=I ** -0.5)
    r = LayerRunner(T, H, I, E, k, moe.MOE_ACT_SWIGLU, gate_up_layout=layout)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    r.route(torch.randn((T, E), generator=g, device="cuda"), idx, w)
    calls = ((r.ws_fwd, lambda: [r.forward(x, idx, w, wgu, wd)]),
             (r.ws_bwd, lambda: r.backward(dy, x, idx, w, wgu, wd)))
    want = [[t.clone() for t in call()] for _, call in calls]
    r.check()
    failed = 0
    for ns in LIMITS_NS:
        for (ws, call), ref in zip(calls, want):
            with_limit(ns, call)
            failed += ended_with_error(ws)
            r.forward(x, idx, w, wgu, wd)      # (the backward takes what a whole forward saved)
            assert all(torch.equal(a, b) for a, b in zip(call(), ref))
    r.check()
    assert failed
