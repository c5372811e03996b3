"""Microscaled 4-bit weights: the codes and scales are determined bit by bit by
the definition (no arithmetic of the quantiser rounds before the code), so they
are compared exactly with a plain restatement in 64 bits."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def exact(w):
    """(codes [E,N,K], scale bytes [E,N,K/32], values [E,K,N]) of w [E,K,N]."""
    E, K, N = w.shape
    b = w.double().transpose(1, 2).reshape(E, N, K // 32, 32)
    amax = b.abs().amax(-1)
    q = torch.full(amax.shape, -127.0, dtype=torch.float64)
    live = amax > 0
    q[live] = torch.ceil(torch.log2(amax[live] / 6.0))
    q = torch.where(live & (6 * torch.exp2(q - 1) >= amax), q - 1, q)
    q = torch.where(live & (6 * torch.exp2(q) < amax), q + 1, q).clamp(-127, 127)
    v = b / torch.exp2(q)[..., None]
    d = (v.abs()[..., None] - GRID).abs()
    # nearest; of two at the same distance the even code
    code = (d + 1e-12 * (torch.arange(8) % 2)).argmin(-1)
    val = GRID[code] * torch.where(torch.signbit(v), -1.0, 1.0) * torch.exp2(q)[..., None]
    code = code + 8 * torch.signbit(v)
    return (code.reshape(E, N, K), (q + 127).to(torch.uint8),
            val.reshape(E, N, K).transpose(1, 2).contiguous())


def unpack(codes):
    c = codes.cpu()
    return torch.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1).long()


def check(w):
    E, K, N = w.shape
    codes, scales = moe.mx_alloc(E, K, N)
    codes.fill_(0xee), scales.fill_(0xee)
    moe.mx_quantize(w.cuda(), codes, scales)
    cx, sx, vx = exact(w)
    assert torch.equal(scales.cpu(), sx)
    assert torch.equal(unpack(codes), cx)
    for dt in (torch.float32, torch.bfloat16):
        back = torch.full((E, K, N), 3.0, dtype=dt, device="cuda")
        moe.mx_dequantize(codes, scales, back)
        # rounded once to the type: only 4 * 2^126 and more leave its range, as infinities
        assert torch.equal(back.cpu(), vx.to(torch.float32).to(dt))


def draw(E, K, N, dt, std=0.02, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((E, K, N), generator=g) * std).to(dt)


@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (2, 64, 64), (3, 416, 200), (1, 288, 72), (2, 256, 128),
                                   (1, 2880, 136), (5, 96, 8)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_round_trip(E, K, N, dt):
    check(draw(E, K, N, dt))


def test_borders_zeros_and_range():
    w = draw(1, 128, 64, torch.float32)
    w[0, :32, 0] = 0
    w[0, :32, 1] = -0.0
    # every border and its neighbours, with a block maximum that gives the scale 1
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat((ties, torch.nextafter(ties, ties * 2), torch.nextafter(ties, ties * 0)))
    w[0, :21, 2], w[0, 21, 2], w[0, 22:32, 2] = near, 6.0, 0.0
    w[0, :21, 3], w[0, 21, 3], w[0, 22:32, 3] = -near, 6.0, 0.0
    w[0, :32, 4] = 6.0                       # amax exactly 6
    w[0, :32, 5] = float(torch.nextafter(torch.tensor(6.0), torch.tensor(7.0)))
    w[0, :32, 6] *= 1e-36
    w[0, :32, 7] *= 1e30
    w[0, 32:64, 0] = torch.finfo(torch.float32).max
    check(w)


def test_tiny_blocks_use_the_smallest_scale():
    w = torch.zeros((1, 32, 8))
    w[0, 3, 0] = 2.0 ** -149                  # below half of the smallest code: 0
    w[0, 3, 1] = 2.0 ** -126                  # 2 * 2^-127
    codes, scales = moe.mx_alloc(1, 32, 8)
    moe.mx_quantize(w.cuda(), codes, scales)
    assert scales.cpu()[0, 0, 0] == 0 and scales.cpu()[0, 1, 0] == 0
    assert unpack(codes)[0, 0].sum() == 0 and unpack(codes)[0, 1, 3] == 4


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_block(bad):
    w = draw(1, 64, 8, torch.bfloat16)
    w[0, 5, 2] = bad
    codes, scales = moe.mx_alloc(1, 64, 8)
    moe.mx_quantize(w.cuda(), codes, scales)
    s = scales.cpu()[0]
    assert s[2, 0] == 255 and int((s == 255).sum()) == 1
    back = torch.empty((1, 64, 8), dtype=torch.bfloat16, device="cuda")
    moe.mx_dequantize(codes, scales, back)
    nan = torch.isnan(back.cpu()[0])
    assert nan[:32, 2].all() and int(nan.sum()) == 32


def test_empty_and_refused():
    codes, scales = moe.mx_alloc(0, 64, 8)
    w = torch.empty((0, 64, 8), device="cuda")
    moe.mx_quantize(w, codes, scales)
    moe.mx_dequantize(codes, scales, w)
    with pytest.raises(ValueError):           # strided weights
        t = torch.zeros((1, 8, 64), device="cuda").transpose(1, 2)
        moe.mx_quantize(t, *moe.mx_alloc(1, 64, 8))
    with pytest.raises(moe.MoeError):         # K not a multiple of 32
        moe.mx_quantize(torch.zeros((1, 40, 8), device="cuda"), *moe.mx_alloc(1, 40, 8))
