"""RMS norm with its outputs over its inputs, where the header allows it: the bits
are those of the call with tensors of its own, in both forms of the kernels (a block
per row, and blocks that walk rows with later rows' copies under way)."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

SIZES = [(20, 288), (1400, 264), (2600, 288), (400, 5152), (320, 8224)]


def rows(T, H, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, H), generator=g, device="cuda").to(dt)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out8", [False, True])
def test_forward(T, H, dt, out8):
    if out8 and H % 32:
        H += 32 - H % 32
    x, res, w = rows(T, H, dt, 1), rows(T, H, dt, 2), rows(1, H, dt, 3)[0]
    y = torch.empty((T, H), dtype=torch.uint8 if out8 else dt, device="cuda")
    ys = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda") if out8 else None
    total = torch.empty_like(x)
    moe.rms_norm_fwd(x, w, y, residual=res, total=total, y_scale=ys)
    for into in (0, 1):
        a = [x.clone(), res.clone()]
        other = torch.empty_like(y)
        ys2 = None if ys is None else torch.empty_like(ys)
        moe.rms_norm_fwd(a[0], w, other, residual=a[1], total=a[into], y_scale=ys2)
        assert torch.equal(a[into], total) and torch.equal(other, y)
        assert ys is None or torch.equal(ys, ys2)
        if not out8:
            a = [x.clone(), res.clone()]
            moe.rms_norm_fwd(a[0], w, a[into], residual=a[1], total=a[1 - into])
            assert torch.equal(a[into], y) and torch.equal(a[1 - into], total)
    if not out8:
        alone, b = torch.empty_like(x), x.clone()
        moe.rms_norm_fwd(x, w, alone)
        moe.rms_norm_fwd(b, w, b)
        assert torch.equal(b, alone)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward(T, H, dt):
    dy, total, d_total, w = rows(T, H, dt, 1), rows(T, H, dt, 2), rows(T, H, dt, 3), rows(1, H, dt, 4)[0]
    rstd = torch.rsqrt(total.float().square().mean(-1))
    ws = moe.rms_norm_workspace(T, H)

    def run(dy, dx, d_total=None):
        dw = torch.empty(H, device="cuda")
        moe.rms_norm_bwd(dy, total, rstd, w, dx, dw, d_total, ws)
        return dx, dw

    for extra in (None, d_total):
        right = run(dy, torch.empty_like(dy), extra)
        over = dy.clone()
        got = run(over, over, extra)
        assert torch.equal(got[0], right[0]) and torch.equal(got[1], right[1])
    over = d_total.clone()
    got = run(dy, over, over)
    assert torch.equal(got[0], right[0]) and torch.equal(got[1], right[1])
