"""4-bit weights of the few-token layer whose blocks differ far in scale: blocks of
zeros (scale byte 0) before, among and after ordinary ones, tiny blocks first, and
the ends of the scales' range.

The bound counts roundings as tests/test_gpu_few.py does (EPS: a step of fp32 for
each addition of an accumulation, K/16 + 64 of them), with the activation's own
rounding to 11 bits: U11, half a step of fp16, of the value, and 2^-31 of its row's
largest activation for the values that a power of two per block leaves fewer bits."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from test_gpu_few import CLAMPED, EPS, SWIGLU, act_and_slopes, make, mx_values, run

pytestmark = pytest.mark.gpu

U11 = torch.finfo(torch.float16).eps / 2
LEFT = 2.0 ** -31


def exact(c):
    """(y, bound on |error|) for 4-bit weights and fp32 output."""
    I, H = c["I"], c["H"]
    y, dy = torch.zeros(c["T"], H, dtype=torch.float64), torch.zeros(c["T"], H, dtype=torch.float64)
    for t in range(c["T"]):
        for j in range(c["k"]):
            e, w = int(c["idx"][t, j]), float(c["w"][t, j])
            h = c["xv"][t] @ c["wgu"][e]
            dh = (H / 16 + 64) * EPS * (c["xv"][t].abs() @ c["wgu"][e].abs())
            a, sg, su = act_and_slopes(h[:I], h[I:], c["act"])
            dg, du = dh[:I], dh[I:]
            da = (sg + 2 * du + 2 * dg) * dg + su * du + 8 * EPS * a.abs()
            da = da + U11 * (a.abs() + da) + LEFT * a.abs().max()
            wd = c["wd"][e].abs()
            o = a @ c["wd"][e]
            y[t] += w * o
            dy[t] += w * (da @ wd + (I / 16 + 64) * EPS * (a.abs() @ wd)) + 40 * EPS * w * o.abs()
    return y, dy


def check(c):
    c["out_fp32"] = True
    c["wgu"], c["wd"] = mx_values(*c["mx"][:2]), mx_values(*c["mx"][2:])
    y, ws = run(c)
    moe.check_device_error(ws)
    ref, bound = exact(c)
    assert torch.isfinite(y).all(), int((~torch.isfinite(y)).sum())
    # (values below fp32's normal range lose bits of their own)
    bad = (y.double() - ref).abs() > bound + 2.0 ** -126
    assert not bad.any(), (int(bad.sum()), float(((y.double() - ref).abs() / (bound + 1e-30)).max()))


def clear(c, which, blocks, columns=slice(None), byte=0):
    """Zeros in these blocks along the contraction, with this scale byte."""
    codes, scales = c["mx"][which], c["mx"][which + 1]
    for b in blocks:
        if b < scales.shape[2]:
            codes[:, columns, 16 * b:16 * b + 16] = 0
            scales[:, columns, b] = byte


SHAPES = [(1, 1088, 1056, 3, 2), (6, 544, 576, 4, 2), (24, 800, 512, 3, 2)]


@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
@pytest.mark.parametrize("which", [0, 2])
@pytest.mark.parametrize("blocks", [[0], [8], [16], [0, 1, 2, 3], [0, 8, 16, 24, 32], list(range(12)), [5, 17]])
def test_zero_blocks(T, H, I, E, k, which, blocks):
    c = make(T, H, I, E, k, SWIGLU, "mx")
    clear(c, which, blocks)
    check(c)
    c = make(T, H, I, E, k, CLAMPED, "mx", seed=1)
    clear(c, which, blocks, slice(0, None, 2))
    check(c)


def test_zero_blocks_of_any_scale():
    for byte in (0, 40, 120, 230, 254):
        c = make(5, 544, 320, 3, 2, SWIGLU, "mx", seed=byte)
        clear(c, 0, [0, 3, 8], byte=byte)
        clear(c, 2, [0, 8], byte=byte)
        check(c)


def test_columns_of_zeros():
    c = make(3, 288, 160, 2, 2, SWIGLU, "mx")
    clear(c, 0, range(9), slice(0, 320, 3))
    clear(c, 2, range(5), slice(1, 288, 4))
    check(c)


@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
@pytest.mark.parametrize("which", [0, 2])
@pytest.mark.parametrize("byte", [1, 5, 20, 40, 80])
def test_tiny_blocks_first(T, H, I, E, k, which, byte):
    """Blocks whose values are not zero but 2^40 to 2^120 below the others'."""
    c = make(T, H, I, E, k, SWIGLU, "mx", seed=byte)
    c["mx"][which + 1][:, ::2, 0:3] = byte
    c["mx"][which + 1][:, 1::3, 8:9] = byte
    check(c)


@pytest.mark.parametrize("T", [2, 20])
def test_scales_that_climb(T):
    """Each step's blocks are larger than all before."""
    c = make(T, 1536, 1280, 2, 1, SWIGLU, "mx")
    for which, first in ((1, 20), (3, 10)):
        s = c["mx"][which]
        climb = torch.linspace(first, 121, s.shape[2]).to(torch.uint8)
        s.copy_(climb.expand_as(s))
    check(c)


def test_tokens_of_zeros_under_the_large_blocks():
    """What the small blocks give is all there is: the large ones meet zeros."""
    c = make(3, 1024, 64, 2, 1, SWIGLU, "mx")
    c["mx"][1][:, :, :16] = 60
    c["mx"][1][:, :, 16:] = 125
    c["x"][:, 512:] = 0
    c["xv"][:, 512:] = 0
    c["x"] *= 2.0 ** 60
    c["xv"] *= 2.0 ** 60
    check(c)


@pytest.mark.parametrize("byte,power", [(238, -108), (250, -125), (254, -126), (30, 95), (10, 110), (120, 0)])
def test_large_scales_by_small_tokens(byte, power):
    """Scales near the ends of their range with tokens that bring the result back."""
    c = make(4, 320, 64, 2, 1, SWIGLU, "mx")
    c["mx"][1].fill_(byte)
    c["x"] = c["xv"].mul(2.0 ** power).to(torch.bfloat16)
    c["xv"] = c["x"].double()
    check(c)


def test_largest_scales():
    """Codes of one half on scales of 2^127, products in range."""
    c = make(1, 64, 32, 1, 1, SWIGLU, "mx")
    c["mx"][1].fill_(112)
    c["mx"][2].fill_(0x11)
    c["mx"][3].fill_(254)
    c["wgu"] = mx_values(*c["mx"][:2])
    check(c)
    assert run(c)[0].abs().max() > 2.0 ** 100


@pytest.mark.parametrize("T", [2, 20])
def test_activation_keeps_11_bits_in_every_block(T):
    """Blocks of activations up to 2^27 below their row's largest: each column of y
    sees one block alone."""
    H, I = 320, 320
    c = make(T, H, I, 1, 1, SWIGLU, "mx", out_fp32=True)
    x = 1.7109375                            # all of bf16's bits
    c["x"].zero_()
    c["x"][:, 0] = x
    c["xv"] = c["x"].double()
    for t in c["mx"][::2]:
        t.zero_()
    c["mx"][0][:, :, 0] = 7                  # 6 for the first value of a token
    c["mx"][1][:, :I] = 130                  # gate: 48 x, where the sigmoid is 1
    c["mx"][3].fill_(127)
    for b in range(I // 32):
        c["mx"][1][:, I + 32 * b:I + 32 * b + 32] = 120 - 3 * b
        c["mx"][2][:, 32 * b:32 * b + 32, 16 * b:16 * b + 16] = 0x52
    c["wgu"], c["wd"] = mx_values(*c["mx"][:2]), mx_values(*c["mx"][2:])
    y, _ = run(c)
    h = c["xv"] @ c["wgu"][0]
    ref = act_and_slopes(h[:, :I], h[:, I:], SWIGLU)[0] @ c["wd"][0]
    # 32 products of one sign, each within 2^-11; sums and the activation within 100 steps
    assert torch.all((y.double() - ref).abs() <= (U11 + 100 * EPS) * ref.abs())
