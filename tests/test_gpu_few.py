"""The expert layer for a few tokens against the definition in 64 bits.

Tolerances count roundings, from the magnitudes that each sum adds up
(u: half a step of bf16, 2^-8; e: a step of fp32, 2^-23, for one addition of an
fp32 accumulation, which the tensor cores may truncate).  A sum of K products
runs over at most K/16 + 64 such additions in one accumulator and across
accumulators:
  dh <= (K/16 + 64) e * sum |x| |W|
  da <= |da/dgate| dgate + |da/dup| dup + u |a|  (bf16 storage rounds a; fp32: 8 e |a|)
  dy <= u |y| + sum_j w (sum da |Wd| + (I/16 + 64) e sum |a| |Wd|) + 40 e sum_j w |o|"""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U, EPS = 2.0 ** -8, 2.0 ** -23
SWIGLU, CLAMPED = moe.MOE_ACT_SWIGLU, moe.MOE_ACT_CLAMPED_GLU


def act_and_slopes(g, u, act, L=7.0, alpha=1.702):
    if act == SWIGLU:
        s = torch.sigmoid(g)
        return g * s * u, (s * (1 + g * (1 - s)) * u).abs(), (g * s).abs()
    gc, uc = g.clamp(max=L), u.clamp(-L, L)
    s = torch.sigmoid(alpha * gc)
    return ((uc + 1) * gc * s, ((uc + 1) * s * (1 + alpha * gc * (1 - s))).abs(), (gc * s).abs())


def mx_values(codes, scales):
    """[E,N,K/2], [E,N,K/32] -> [E,K,N] in 64 bits."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=torch.float64)
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1)
    v = v.reshape(*scales.shape, 32) * torch.exp2(scales.double() - 127)[..., None]
    return v.reshape(*codes.shape[:-1], -1).transpose(1, 2)


def make(T, H, I, E, k, act, weights="bf16", bias=False, x8=False, il=False, out_fp32=False, seed=0,
         idx=None, w_std=0.05):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = torch.float32 if weights == "fp32" else torch.bfloat16
    c = dict(T=T, H=H, I=I, E=E, k=k, act=act, weights=weights, il=il, out_fp32=out_fp32, dt=dt)
    x = rn(T, H)
    if x8:
        b = x.view(T, H // 32, 32)
        q = torch.ceil(torch.log2(b.abs().amax(-1) / 448)).clamp(-127, 127)
        c["x"] = (b / torch.exp2(q)[..., None]).to(torch.float8_e4m3fn).view(T, H)
        c["x_scale"] = (q + 127).to(torch.uint8)
        c["xv"] = (c["x"].double().view(T, H // 32, 32) * torch.exp2(q.double())[..., None]).view(T, H)
    else:
        c["x"] = x.to(dt)
        c["xv"] = c["x"].double()
    if idx is None:
        idx = torch.topk(rn(T, E), k, dim=-1).indices
    c["idx"] = idx.to(torch.int32).contiguous()
    c["w"] = torch.softmax(rn(T, k), -1)
    if weights == "mx":
        rb = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
        c["mx"] = (rb(0, 256, E, 2 * I, H // 2), rb(118, 123, E, 2 * I, H // 32),
                   rb(0, 256, E, H, I // 2), rb(118, 123, E, H, I // 32))
        c["wgu"], c["wd"] = mx_values(*c["mx"][:2]), mx_values(*c["mx"][2:])
    else:
        c["w_gate_up"], c["w_down"] = (w_std * rn(E, H, 2 * I)).to(dt), (w_std * rn(E, I, H)).to(dt)
        c["wgu"], c["wd"] = c["w_gate_up"].double(), c["w_down"].double()
    if bias:
        c["bgu"], c["bd"] = (0.5 * rn(E, 2 * I)).to(dt), (0.5 * rn(E, H)).to(dt)
    return c


def exact(c):
    """(y, bound on |error|)."""
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    y, dy = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e, w = int(c["idx"][t, j]), float(c["w"][t, j])
            if e < 0 or e >= c["E"]:
                continue
            h = c["xv"][t] @ c["wgu"][e]
            dh = (H / 16 + 64) * EPS * (c["xv"][t].abs() @ c["wgu"][e].abs())
            if "bgu" in c:
                h = h + c["bgu"][e].double()
                dh = dh + EPS * h.abs()
            gate, up = (h[0::2], h[1::2]) if c["il"] else (h[:I], h[I:])
            dg, du = (dh[0::2], dh[1::2]) if c["il"] else (dh[:I], dh[I:])
            a, sg, su = act_and_slopes(gate, up, c["act"])
            # second order: the slopes move with dg and du by at most 2 each per unit
            da = (sg + 2 * du + 2 * dg) * dg + su * du + 8 * EPS * a.abs()
            if c["weights"] != "fp32":
                da = da + U * (a.abs() + da)
            o = a @ c["wd"][e]
            do = da @ c["wd"][e].abs() + (I / 16 + 64) * EPS * (a.abs() @ c["wd"][e].abs())
            if "bd" in c:
                o = o + c["bd"][e].double()
            y[t] += w * o
            dy[t] += w * do + 40 * EPS * w * o.abs()
    if c["weights"] != "fp32" and not c["out_fp32"]:
        dy = dy + U * (y.abs() + dy)
    return y, dy


def run(c, ws=None, stream=None):
    s = moe.Shape(c["T"], c["H"], c["I"], c["E"], c["k"], c["act"],
                  moe.MOE_FP32 if c["weights"] == "fp32" else moe.MOE_BF16, 7.0, 1.702,
                  1 if c["il"] else 0, c["out_fp32"])
    d = {n: (tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda())
         for n, v in c.items() if isinstance(v, (torch.Tensor, tuple)) and n not in ("wgu", "wd", "xv")}
    ws = moe.few_workspace(s) if ws is None else ws
    y = torch.full((c["T"], c["H"]), 77.0, device="cuda",
                   dtype=torch.float32 if c["out_fp32"] else c["dt"])
    mx = moe.mx_struct(*d["mx"]) if "mx" in d else None
    for _ in range(2):       # the workspace is left ready for the next call
        moe.ffn_few(s, d["x"], d["idx"], d["w"], d.get("w_gate_up"), d.get("w_down"), y, ws,
                    bias=moe.bias_struct(d.get("bgu"), d.get("bd")), x_scale=d.get("x_scale"), mx=mx,
                    stream=stream)
    torch.cuda.synchronize()
    return y.cpu(), ws


def check(c):
    y, ws = run(c)
    moe.check_device_error(ws)
    ref, bound = exact(c)
    bad = (y.double() - ref).abs() > bound + 1e-30
    assert not bad.any(), (int(bad.sum()), float(((y.double() - ref).abs() / (bound + 1e-30)).max()))


SIZES = [(1, 8, 8, 1, 1), (1, 128, 128, 8, 2), (2, 136, 72, 5, 3), (5, 264, 200, 16, 4),
         (8, 64, 520, 3, 2), (9, 200, 264, 4, 4), (17, 512, 136, 40, 8), (33, 96, 64, 2, 2),
         (64, 320, 96, 7, 3), (128, 72, 40, 9, 4)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("weights,act,bias,il", [("bf16", SWIGLU, False, False), ("bf16", CLAMPED, True, True),
                                                 ("fp32", SWIGLU, True, False), ("fp32", CLAMPED, False, True)])
def test_dense_weights(T, H, I, E, k, weights, act, bias, il):
    check(make(T, H, I, E, k, act, weights, bias=bias, il=il))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 32, 32, 1, 1), (1, 128, 96, 8, 2), (3, 288, 160, 5, 3),
                                       (9, 64, 416, 4, 4), (17, 512, 128, 20, 8), (40, 96, 64, 2, 2),
                                       (128, 64, 32, 9, 4)])
@pytest.mark.parametrize("act,bias,il,x8", [(SWIGLU, False, False, False), (CLAMPED, True, True, True),
                                            (CLAMPED, False, False, True)])
def test_microscaled_weights(T, H, I, E, k, act, bias, il, x8):
    check(make(T, H, I, E, k, act, "mx", bias=bias, il=il, x8=x8))


@pytest.mark.parametrize("weights", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 12])
def test_8bit_tokens_with_dense_weights(T, weights):
    check(make(T, 320, 72, 6, 3, SWIGLU, weights, x8=True))


@pytest.mark.parametrize("weights", ["bf16", "mx", "fp32"])
def test_one_expert_takes_all_and_repeats(weights):
    check(make(50, 64, 64, 4, 2, SWIGLU, weights, idx=torch.full((50, 2), 2)))
    check(make(7, 64, 64, 4, 3, SWIGLU, weights, idx=torch.tensor([[1, 1, 3]] * 7)))


def test_many_experts_and_choices():
    check(make(4, 64, 40, 1024, 32, CLAMPED))
    check(make(128, 32, 32, 1024, 32, SWIGLU, "mx"))


def test_fp32_output():
    check(make(3, 264, 136, 8, 4, CLAMPED, bias=True, out_fp32=True))
    check(make(20, 256, 128, 8, 4, SWIGLU, "mx", out_fp32=True))


def test_model_size_one_token():
    check(make(1, 2880, 2880, 6, 4, CLAMPED, bias=True, w_std=0.02))
    check(make(1, 2880, 2880, 6, 4, CLAMPED, "mx", bias=True, x8=True))


@pytest.mark.parametrize("byte", [0, 1, 60, 128, 129, 200, 254])
def test_every_scale(byte):
    """Scales that need a second product, and weights below bf16's normal range."""
    c = make(1, 64, 32, 1, 1, SWIGLU, "mx")
    c["mx"][1].fill_(127)
    c["mx"][3].fill_(byte)
    # large scales: codes of one half, small ones: of 6, so that y stays in range
    if byte > 250:
        c["mx"][2].fill_(0x11)
        c["xv"] *= 0.0
        c["x"].zero_()
    c["wgu"], c["wd"] = mx_values(*c["mx"][:2]), mx_values(*c["mx"][2:])
    c["out_fp32"] = True
    y, _ = run(c)
    ref, bound = exact(c)
    # results below fp32's normal range lose bits of their own
    assert torch.all((y.double() - ref).abs() <= bound + 2.0 ** -126)


def test_nan_scale_reaches_its_columns_only():
    c = make(2, 64, 32, 2, 1, SWIGLU, "mx", idx=torch.tensor([[0], [1]]))
    c["mx"][3][1, 5, 0] = 255
    y, _ = run(c)
    nan = torch.isnan(y)
    assert nan[1, 5] and int(nan.sum()) == 1


def test_non_finite_tokens_stay_apart():
    c = make(6, 64, 64, 3, 2, CLAMPED)
    c["x"][2, 7] = float("nan")
    y, _ = run(c)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("T,H,I,E,k", [(5, 96, 352, 6, 2), (30, 1056, 288, 4, 2), (24, 416, 544, 3, 2),
                                       (2, 2080, 736, 12, 4)])
def test_microscaled_odd_blocks_and_wide_scales(T, H, I, E, k):
    """Contractions that end inside a step, odd counts of blocks, and scales far from
    their column's first one."""
    check(make(T, H, I, E, k, SWIGLU, "mx", bias=True))
    c = make(T, H, I, E, k, CLAMPED, "mx", x8=True, seed=1)
    g = torch.Generator().manual_seed(2)
    for s in (c["mx"][1], c["mx"][3]):
        s.copy_(torch.randint(100, 128, s.shape, generator=g))
    c["wgu"], c["wd"] = mx_values(*c["mx"][:2]), mx_values(*c["mx"][2:])
    check(c)


def test_microscaled_scales_at_odd_addresses():
    c = make(20, 128, 320, 6, 2, SWIGLU, "mx")
    a, _ = run(c)
    s = moe.Shape(20, 128, 320, 6, 2, SWIGLU, moe.MOE_BF16, 7.0, 1.702, 0, 0)
    d = [v.cuda() for v in c["mx"]]
    for i in (1, 3):
        odd = torch.empty(d[i].numel() + 1, dtype=torch.uint8, device="cuda")[1:]
        odd.copy_(d[i].flatten())
        d[i] = odd.view(d[i].shape)
        assert d[i].data_ptr() % 2 == 1
    y = torch.empty(20, 128, device="cuda", dtype=torch.bfloat16)
    moe.ffn_few(s, c["x"].cuda(), c["idx"].cuda(), c["w"].cuda(), None, None, y, moe.few_workspace(s),
                mx=moe.mx_struct(*d))
    assert torch.equal(y.cpu(), a)


@pytest.mark.parametrize("T,H,I", [(6, 64, 64), (6, 352, 96), (20, 96, 288)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_stay_apart_on_4_bits(T, H, I, bad):
    c = make(T, H, I, 3, 2, SWIGLU, "mx")
    c["x"][2, 7] = bad
    y, _ = run(c)
    others = [t for t in range(T) if t != 2]
    assert torch.isnan(y[2]).all() and torch.isfinite(y[others]).all()


@pytest.mark.parametrize("mx", [True, False])
def test_experts_past_32_bits(mx):
    """The last of many experts gives the bits that it gives alone."""
    H, I, E = (4096, 4096, 300) if mx else (2048, 2048, 300)
    g = torch.Generator("cuda").manual_seed(3)
    if mx:
        one = [torch.randint(0, 256, (1, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
               for n, k in ((2 * I, H), (H, I))]
        one = [one[0], torch.randint(118, 122, (1, 2 * I, H // 32), generator=g, device="cuda", dtype=torch.uint8),
               one[1], torch.randint(118, 122, (1, H, I // 32), generator=g, device="cuda", dtype=torch.uint8)]
    else:
        one = [0.02 * torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
               for s in ((1, H, 2 * I), (1, I, H))]
    x = torch.randn((3, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.ones((3, 1), device="cuda")
    out = []
    for n in (1, E):
        ts = []
        for t in one:
            big = torch.empty((n,) + t.shape[1:], dtype=t.dtype, device="cuda")
            big[n - 1] = t[0]
            ts.append(big)
        s = moe.Shape(3, H, I, n, 1, SWIGLU)
        idx = torch.full((3, 1), n - 1, dtype=torch.int32, device="cuda")
        y = torch.empty((3, H), dtype=torch.bfloat16, device="cuda")
        moe.ffn_few(s, x, idx, w, None if mx else ts[0], None if mx else ts[1], y, moe.few_workspace(s),
                    mx=moe.mx_struct(*ts) if mx else None)
        out.append(y.cpu())
    assert max(t.numel() * t.element_size() for t in ts) > 2 ** 32
    assert torch.isfinite(out[0]).all() and torch.equal(*out)


def test_bad_ids_are_reported_and_left_out():
    idx = torch.tensor([[0, 9], [-1, 1], [2, 3]])
    c = make(3, 64, 64, 4, 2, SWIGLU, idx=idx)
    y, ws = run(c)
    with pytest.raises(moe.MoeError) as e:
        moe.check_device_error(ws)
    assert e.value.status == moe.MOE_ERR_BAD_INDEX
    ref, bound = exact(c)
    assert torch.all((y.double() - ref).abs() <= bound)
    c = make(3, 64, 64, 4, 2, SWIGLU, idx=torch.full((3, 2), 4))
    assert torch.all(run(c)[0] == 0)


def test_wait_limit_unwinds():
    """A limit of 1 ns on the waits for the codes' copies suffices or is reported, and
    the next call on the same workspace with the usual limit is right."""
    c = make(24, 1056, 736, 12, 2, SWIGLU, "mx")
    s = moe.Shape(24, 1056, 736, 12, 2, SWIGLU, moe.MOE_BF16, 7.0, 1.702, 0, 0)
    right, ws = run(c)
    d = [c[n].cuda() for n in ("x", "idx", "w")]
    mx = [t.cuda() for t in c["mx"]]
    y = torch.empty(24, 1056, device="cuda", dtype=torch.bfloat16)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    flush.zero_()             # the codes are not in the L2 cache
    torch.cuda.synchronize()
    old = moe.moe_set_wait_timeout_ns(1)
    try:
        moe.ffn_few(s, *d, None, None, y, ws, mx=moe.mx_struct(*mx))
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_timeout_ns(old)
    try:                      # (the hardware's own wait may be long enough)
        moe.check_device_error(ws)
        assert torch.equal(y.cpu(), right)
    except moe.MoeError as e:
        assert e.status == moe.MOE_ERR_TIMEOUT
    ws[:4] = 0
    moe.ffn_few(s, *d, None, None, y, ws, mx=moe.mx_struct(*mx))
    moe.check_device_error(ws)
    assert torch.equal(y.cpu(), right)


def test_agrees_with_the_layer_for_many_tokens():
    from dispatch_gemm_combine_gb300.runner import LayerRunner
    c = make(16, 256, 128, 8, 2, SWIGLU)
    r = LayerRunner(16, 256, 128, 8, 2, SWIGLU, training=False, backward=False)
    args = [c[n].cuda() for n in ("x", "idx", "w", "w_gate_up", "w_down")]
    y = r.forward(*args, use_plan=False)
    y = y.clone()
    few = r.few(*args)
    _, bound = exact(c)
    # each of the two is within the bound (the other layer's products are tensor-core sums too)
    assert torch.all((y.double() - few.double()).abs().cpu() <= 2 * bound)


def test_repeatable_on_streams_and_in_a_graph():
    c = make(13, 512, 264, 20, 4, SWIGLU, bias=True)
    a, ws = run(c)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b, _ = run(c)
    assert torch.equal(a, b)
    shape = moe.Shape(13, 512, 264, 20, 4, SWIGLU)
    d = [c[n].cuda() for n in ("x", "idx", "w", "w_gate_up", "w_down")]
    bias = [c[n].cuda() for n in ("bgu", "bd")]
    y = torch.zeros((13, 512), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.ffn_few(shape, *d, y, ws, bias=moe.bias_struct(*bias))
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), a)


def test_refusals():
    c = make(2, 64, 64, 4, 2, SWIGLU)
    s = moe.Shape(2, 64, 64, 4, 2, SWIGLU)
    d = [c[n].cuda() for n in ("x", "idx", "w", "w_gate_up", "w_down")]
    y, ws = torch.empty((2, 64), dtype=torch.bfloat16, device="cuda"), moe.few_workspace(s)
    with pytest.raises(ValueError):
        moe.ffn_few(s, d[0].t().contiguous().t(), *d[1:], y, ws)
    with pytest.raises(ValueError):
        moe.ffn_few(s, d[0].float(), *d[1:], y, ws)
    with pytest.raises(ValueError):
        moe.ffn_few(s, d[0], d[1].long(), *d[2:], y, ws)
    with pytest.raises(moe.MoeError):
        moe.ffn_few(s, d[0], d[1], d[2], None, None, y, ws)
    with pytest.raises(moe.MoeError):
        moe.few_workspace(moe.Shape(129, 64, 64, 4, 2))
    e = moe.Shape(0, 64, 64, 4, 2)
    moe.ffn_few(e, d[0][:0], d[1][:0], d[2][:0], d[3], d[4], y[:0], moe.few_workspace(e))
