"""RMS norm (with the residual's addition and the 8-bit output) and its
gradient against the definitions in 64 bits.

Tolerances count roundings.  u is half a step of the type relative to the value
(finfo.eps / 2).  An output is rounded once to its type (u); before that the
fp32 arithmetic makes a handful of roundings of u32 each, plus those of the sum
over the row, which stay below (8 + log2 terms + warps) < 64 of them.  The
e4m3 codes may fall on either side of a border where the fp32 value does: one
code step there, none elsewhere."""

import numpy as np
import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def draw(T, H, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, H), generator=g) * std).to(dt)


def exact_fwd(x, res, w, eps):
    r = x.double() + (res.double() if res is not None else 0)
    rs = 1 / torch.sqrt(r.square().mean(-1) + eps)
    return r, rs, r * rs[:, None] * w.double()


def check_fwd(T, H, dt, res, out8, eps=1e-6, std=1.0, x=None):
    x = draw(T, H, dt, 1, std) if x is None else x
    r = draw(T, H, dt, 2, 3 * std) if res else None
    w = (1 + 0.1 * draw(1, H, torch.float32, 3)[0]).to(dt)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = torch.empty((T, H), dtype=torch.uint8 if out8 else dt, device="cuda")
    ys = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda") if out8 else None
    total = torch.empty((T, H), dtype=dt, device="cuda")
    rstd = torch.empty(T, device="cuda")
    moe.rms_norm_fwd(x.cuda(), dev(w), y, eps, dev(r), total, rstd, ys)
    rx, rs, yx = exact_fwd(x, r, w, eps)
    assert torch.all((total.cpu().double() - rx).abs() <= (half_step(dt) + U32) * rx.abs())
    # rs: the sum's roundings halve in the root
    assert torch.all((rstd.cpu().double() - rs).abs() <= 40 * U32 * rs)
    if not out8:
        bound = (half_step(dt) + 48 * U32) * yx.abs() + 1e-40
        assert torch.all((y.cpu().double() - yx).abs() <= bound)
        return
    b = yx.view(T, -1, 32)
    amax = b.abs().amax(-1)
    scale = torch.exp2(ys.cpu().double() - 127)
    # the smallest power of two with amax <= 448 scale, up to the fp32 error of amax
    slack = 48 * U32
    live = amax > 0
    assert torch.all((448 * scale >= amax * (1 - slack))[live])
    assert torch.all((224 * scale <= amax * (1 + slack))[live])
    assert torch.all(ys.cpu()[~live] == 0)
    code = y.cpu().view(torch.float8_e4m3fn).double().view(T, -1, 32)
    v = b / scale[..., None]
    # half a step of e4m3: 2^-4 of the value's power of two, at least half of 2^-9
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    assert torch.all((code - v).abs() <= 0.5 * step + 48 * U32 * v.abs() + 448 * slack * (v.abs() > 440))


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2880), (3, 32), (5, 2880), (7, 4096), (33, 264),
                                 (2, 8192), (2, 8200), (3, 16384), (2, 32768), (513, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward(T, H, dtype):
    check_fwd(T, H, DT[dtype], True, False)
    check_fwd(T, H, DT[dtype], False, False)


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2880), (5, 4096), (9, 96), (2, 8192), (2, 16384), (2, 32768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_8bit(T, H, dtype):
    check_fwd(T, H, DT[dtype], True, True)
    check_fwd(T, H, DT[dtype], False, True)


@pytest.mark.parametrize("T,H,out8", [(1400, 288, True), (700, 2912, True), (400, 5152, True), (320, 8224, True),
                                      (400, 5128, False), (320, 8200, False), (1400, 264, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_several_rows_per_block(T, H, out8, dtype):
    """More rows than resident blocks, and warps that a row's end cuts."""
    check_fwd(T, H, DT[dtype], True, out8)
    check_fwd(T, H, DT[dtype], False, out8)


def test_small_and_large_rows():
    check_fwd(4, 256, torch.float32, False, False, std=1e-12)
    check_fwd(4, 256, torch.float32, False, False, std=1e15)
    x = draw(4, 256, torch.bfloat16, 5)
    x[1] = 0
    x[2, 32:] = 0
    check_fwd(4, 256, torch.bfloat16, False, False, x=x)
    check_fwd(4, 256, torch.bfloat16, False, True, x=x)


def test_non_finite_rows_stay_apart():
    x = draw(4, 64, torch.bfloat16, 6)
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")
    y8 = torch.empty((4, 64), dtype=torch.uint8, device="cuda")
    ys = torch.empty((4, 2), dtype=torch.uint8, device="cuda")
    moe.rms_norm_fwd(x.cuda(), w, y)
    moe.rms_norm_fwd(x.cuda(), w, y8, y_scale=ys)
    y, ys = y.cpu().float(), ys.cpu()
    assert torch.isnan(y[1]).all()
    # 1 / inf = 0: the other values of that row are 0, the infinite one is NaN
    assert torch.isnan(y[2, 40]) and torch.all(torch.cat((y[2, :40], y[2, 41:])) == 0)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert ys[1].tolist() == [255, 255] and ys[2].tolist() == [0, 255]
    assert 255 not in ys[0].tolist() + ys[3].tolist()


def run_bwd(T, H, dt, d_total, seed=11, frozen=False):
    total = draw(T, H, dt, seed, 3.0)
    dy, dt_ = draw(T, H, dt, seed + 1), (draw(T, H, dt, seed + 2) if d_total else None)
    w = (1 + 0.1 * draw(1, H, torch.float32, seed + 3)[0]).to(dt)
    rstd = torch.rsqrt(total.double().square().mean(-1) + 1e-6).float()
    dx = torch.empty((T, H), dtype=dt, device="cuda")
    dw = None if frozen else torch.empty(H, device="cuda")
    ws = None if frozen else moe.rms_norm_workspace(T, H)
    moe.rms_norm_bwd(dy.cuda(), total.cuda(), rstd.cuda(), w.cuda(), dx, dw,
                     None if dt_ is None else dt_.cuda(), ws)
    return total, dy, dt_, w, rstd, dx.cpu(), None if frozen else dw.cpu()


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2880), (3, 32), (700, 2880), (65, 4096), (33, 264),
                                 (5, 8200), (3, 16384), (2, 32768), (2049, 128)])
@pytest.mark.parametrize("dtype,d_total", [("bf16", True), ("bf16", False), ("fp32", True)])
def test_backward(T, H, dtype, d_total):
    dt = DT[dtype]
    total, dy, dt_, w, rstd, dx, dw = run_bwd(T, H, dt, d_total)
    xh = total.double() * rstd.double()[:, None]
    n = dy.double() * w.double()
    inner = n - xh * (n * xh).mean(-1, keepdim=True)
    ref = rstd.double()[:, None] * inner
    # what the fp32 roundings act on: the terms before they cancel
    mag = rstd.double()[:, None] * (n.abs() + xh.abs() * (n * xh).abs().mean(-1, keepdim=True))
    if dt_ is not None:
        ref, mag = ref + dt_.double(), mag + dt_.double().abs()
    assert torch.all((dx.double() - ref).abs() <= half_step(dt) * ref.abs() + 64 * U32 * mag + 1e-40)
    terms = dy.double() * xh
    # fp32 sums of T terms: at most rows per block + 64 additions, each u32 of the partial sum
    rows = -(-T // 152) + 64
    assert torch.all((dw.double() - terms.sum(0)).abs() <= (rows + 4) * U32 * terms.abs().sum(0) + 1e-40)


@pytest.mark.parametrize("T,H", [(2600, 264), (1400, 2888), (400, 5128), (320, 8200)])
@pytest.mark.parametrize("dtype,d_total", [("bf16", True), ("fp32", False), ("fp32", True)])
def test_backward_several_rows_per_block(T, H, dtype, d_total):
    test_backward(T, H, dtype, d_total)


def test_backward_against_differences():
    """<dx, d> is the directional derivative of <dy, y>, by central differences
    of the 64-bit definition; likewise for the weight."""
    T, H = 6, 96
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=g)
    w = 1 + 0.1 * torch.randn(H, generator=g)
    dy = torch.randn((T, H), generator=g)
    d = torch.randn((T, H), generator=g).double()
    dwd = torch.randn(H, generator=g).double()
    y = torch.empty((T, H), device="cuda")
    total, rstd = torch.empty((T, H), device="cuda"), torch.empty(T, device="cuda")
    moe.rms_norm_fwd(x.cuda(), w.cuda(), y, 1e-5, None, total, rstd)
    dx, dw = torch.empty((T, H), device="cuda"), torch.empty(H, device="cuda")
    moe.rms_norm_bwd(dy.cuda(), total, rstd, w.cuda(), dx, dw, ws=moe.rms_norm_workspace(T, H))

    def f(xv, wv):
        return (dy.double() * exact_fwd(xv, None, wv, 1e-5)[2]).sum()

    h = 1e-5
    num_x = (f(x.double() + h * d, w.double()) - f(x.double() - h * d, w.double())) / (2 * h)
    num_w = (f(x.double(), w.double() + h * dwd) - f(x.double(), w.double() - h * dwd)) / (2 * h)
    # fp32 gradients: 64 u32 of the sum of magnitudes; the differences' own error is ~h^2
    mag = (dx.cpu().double() * d).abs().sum()
    assert abs((dx.cpu().double() * d).sum() - num_x) <= 64 * U32 * mag + 1e-7 * mag
    magw = (dw.cpu().double() * dwd).abs().sum()
    assert abs((dw.cpu().double() * dwd).sum() - num_w) <= 64 * U32 * magw + 1e-7 * magw


def test_frozen_weight_and_repeatable():
    a = run_bwd(300, 2880, torch.bfloat16, True)
    b = run_bwd(300, 2880, torch.bfloat16, True)
    c = run_bwd(300, 2880, torch.bfloat16, True, frozen=True)
    assert torch.equal(a[5], b[5]) and torch.equal(a[6], b[6]) and torch.equal(a[5], c[5])


def test_in_place_and_other_stream_and_graph():
    T, H = 20, 512
    x, r = draw(T, H, torch.bfloat16, 1).cuda(), draw(T, H, torch.bfloat16, 2).cuda()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, total = torch.empty_like(x), torch.empty_like(x)
    moe.rms_norm_fwd(x, w, y, residual=r, total=total)
    torch.cuda.synchronize()
    x2, r2 = x.clone(), r.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.rms_norm_fwd(x2, w, x2, residual=r2, total=r2)      # y over x, total over residual
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(r2, total)


def test_empty():
    H = 64
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    moe.rms_norm_fwd(e, w, e)
    dw = torch.full((H,), 7.0, device="cuda")
    moe.rms_norm_bwd(e, e, torch.empty(0, device="cuda"), w, e, dw, ws=moe.rms_norm_workspace(0, H))
    assert np.all(dw.cpu().numpy() == 0)
