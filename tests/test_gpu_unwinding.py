"""Waits that run out at any place of a pair's ring: each CTA of a pair waits by its own
clock, so one may have given up where the other has loaded on.  The call ends, its
error is reported (or its result is right), and the next call on the same workspace is
right.  Limits from one that no wait keeps to one that most do."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

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
