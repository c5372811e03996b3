"""Orthogonal updates by Newton-Schulz products, against the iteration in 64 bits.

Two comparisons.  `emulated` computes in 64 bits but rounds where the kernels round to
fp16 (x_0, and each step's a, b and x, all held with the same power of two; b not for at
most 128 rows, where it is held as two fp16 values, 2^-22 of it left out): what is left between the two is the fp32 accumulation, which tips one rounding in some hundred
the other way, and the output's rounding to bf16, off by at most u = 2^-8 of a value
and 0.6 u in the 2-norm (a rounding's error is spread over half a step).  The bound is
u of the 2-norm, so 0.4 u = 1.6e-3 is left for tipped roundings: a tenth of all
roundings tipped by a whole step (2^-10) and amplified tenfold stays below it.
`exact` rounds nowhere.  The 16 roundings of five steps have at most
2^-11 / sqrt(3) = 2.8e-4 in the 2-norm; a rounding of a is amplified by up to
|c1| s^2 + 2 |c2| s^4 = 15 at s = 1.2, the others less, so their root sum of squares
is below 4 * 15 * 2.8e-4 = 1.7e-2 (the worst case, all steps at s = 1.2)."""

import math

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
COEFS = (3.4445, -4.7750, 2.0315)


def start(g, eps):
    x = g.double()
    return x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps).clamp(min=1e-300)


def exact(g, steps=5, coefs=None, eps=1e-7):
    x = start(g, eps)
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT if flip else x
    for i in range(steps):
        c = (coefs or [COEFS] * steps)[i]
        a = x @ x.mT
        x = c[0] * x + (c[1] * a + c[2] * (a @ a)) @ x
    return x.mT if flip else x


def emulated(g, steps=5, coefs=None, eps=1e-7):
    x = start(g, eps)
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT if flip else x
    h = lambda t: t.to(torch.float16).double()  # noqa: E731
    S = 2.0 ** min(round(math.log2(x.shape[-1]) / 2), 6)
    x = h(x * S)
    eye = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device)
    for i in range(steps):
        c = (coefs or [COEFS] * steps)[i]
        a = h(x @ x.mT)
        b = c[0] * S * S * eye + c[1] * a + c[2] / (S * S) * (a @ a)
        b = b if x.shape[-2] <= 128 else h(b)
        x = b @ x / (S * S)
        x = h(x) if i + 1 < steps else x
    x = x / S
    return x.mT if flip else x


def rel(got, want):
    """The largest relative error of a matrix in the 2-norm."""
    d = (got.double() - want).square().sum((-2, -1)).sqrt()
    n = want.square().sum((-2, -1)).sqrt()
    return float(torch.where(n > 0, d / n.clamp(min=1e-300), d).max())


def draw(shape, dt, seed=1, std=0.01):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def run(g, out=None, ws=None, **kw):
    out = torch.full(g.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = moe.orthogonalize_workspace(g) if ws is None else ws
    moe.orthogonalize(g, out, ws, **kw)
    moe.check_device_error(ws)
    return out


def check(g, **kw):
    out = run(g, **kw)
    kw.pop("ws", None)
    scale = kw.pop("scale", 1.0)
    assert rel(out, scale * emulated(g, **kw)) <= U
    assert rel(out, scale * exact(g, **kw)) <= U + 1.7e-2
    return out


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 5), (16, 16), (8, 200), (64, 64), (65, 63), (128, 128), (129, 127), (128, 300), (300, 128),
          (257, 255), (255, 513), (256, 256), (512, 512), (640, 384), (1000, 40), (40, 1001), (511, 1029), (2880, 128), (100, 512), (513, 33), (128, 2049), (4096, 72), (24, 4097), (1, 5000), (4100, 3), (130, 20000)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shapes(M, N, dtype):
    check(draw((M, N), dtype))
    check(draw((3, M, N), dtype, 2))


def test_large_matrix():
    check(draw((1500, 2300), torch.float32))


def test_more_matrices_than_a_launch_takes():
    check(draw((1301, 24, 16), torch.float32))


@pytest.mark.parametrize("E,M,N", [(5, 33, 900), (9, 1500, 97), (20, 128, 1100), (9, 2880, 47), (40, 100, 250), (2, 128, 4096)])
def test_clusters_in_waves(E, M, N):
    """Narrow matrices on clusters, more of them than fit at once."""
    check(draw((E, M, N), torch.bfloat16))


def test_singular_values_and_vectors():
    """Of a matrix with known singular values: the result has its vectors."""
    q = lambda n, s: torch.linalg.qr(torch.randn((n, 96), generator=torch.Generator().manual_seed(s), dtype=torch.float64))[0]  # noqa: E731
    u, v = q(200, 1), q(160, 2)
    s = torch.linspace(0.2, 1.0, 96, dtype=torch.float64)
    g = (u * s @ v.t()).float().cuda()
    out = run(g).cpu().double()
    core = u.t() @ out @ v
    # five steps bring [0.02, 0.2] (s over the Frobenius norm) into [0.68, 1.21]
    assert torch.all((core.diagonal() > 0.66) & (core.diagonal() < 1.23))
    off = core - torch.diag(core.diagonal())
    assert off.norm() <= (U + 1.7e-2) * core.norm()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-12, 1e12, 1e30, 1e37])
def test_scales_of_the_input(scale):
    g = draw((2, 70, 130), torch.float32, std=1.0)
    want = run(g, eps=0.0)
    got = run(g * scale, eps=0.0)
    assert rel(got, exact(g * scale, eps=0.0)) <= U + 1.7e-2
    assert rel(got, want.double()) <= 2 * U
    if scale < 1e-10:
        # eps on a small norm: x_0 is small, and grows by c0 a step
        check(g * scale, eps=float((g * scale).double().norm()) * 3)


def test_zeros_and_non_finite_matrices_stay_apart():
    for shape in ((5, 40, 72), (5, 300, 200)):
        g = draw(shape, torch.float32)
        g[1] = 0
        g[2, 3, 5] = float("nan")
        g[3, 0, 0] = float("inf")
        for eps in (0.0, 1e-7):
            out = run(g, eps=eps)
            assert not out[1].any()
            assert torch.isnan(out[2:4]).all()
            assert rel(out[::4], exact(g[::4], eps=eps)) <= U + 1.7e-2


@pytest.mark.parametrize("M,N", [(70, 130), (300, 200)])
def test_norms_far_below_eps(M, N):
    """x_0 = g / (|g| + eps) is small, not NaN, where eps leaves fp32's range beside the
    norm (scaled by 2^80 for matrices below 2^-20)."""
    g = draw((2, M, N), torch.float32, std=1e-12)
    check(g, eps=float(g.double().square().sum((-2, -1)).sqrt().max()) * 100)
    for eps in (1e15, 1e20, 3e38):
        assert not run(g, eps=eps).any()
    g[1, 3, 4] = float("nan")
    out = run(g, eps=1e20)
    assert not out[0].any() and torch.isnan(out[1]).all()


def test_small_scales():
    """The least scale: out is a bf16 normal number's size, fp32 holds scale / S^3."""
    g = draw((2, 70, 130), torch.float32)
    check(g, scale=2.0 ** -100)
    check(draw((2, 200, 130), torch.float32), scale=-2.0 ** -100)
    assert not run(g, scale=0.0).any()


def test_rank_one_and_equal_rows():
    """Where g has one singular value, what the roundings of x leave beside its
    direction grows by c0 a step: a rounding of x_j (2.8e-4 of its norm, which is at
    most 1.22 times the result's over 0.68) by c0^(5 - j), their sum is below
    2.8e-4 * 1.8 * 682 = 0.35 of the result.  Along the direction nothing grows."""
    for u, v in ((draw((90, 1), torch.float32, 3, 1.0), draw((1, 130), torch.float32, 4, 1.0)),
                 (torch.ones((40, 1), device="cuda"), torch.ones((1, 50), device="cuda"))):
        g = u @ v
        out, want = run(g).double(), exact(g)
        along = u.double() @ (u.double().t() @ out @ v.double().t()) @ v.double() / (u.double().norm() * v.double().norm()) ** 2
        assert rel(along, want) <= U + 1.7e-2
        assert rel(out, want) <= 0.35 + U
    check(torch.eye(48, device="cuda"))


@pytest.mark.parametrize("M,N", [(72, 200), (300, 136), (133, 77)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0, 1, 8])
def test_strided_views(M, N, dtype, first):
    """Columns of wider tensors, rows and matrices apart, at odd addresses; what lies
    beside the result stays."""
    wide = draw((3, M + 2, N + 24), dtype)
    g = wide[:, 1:M + 1, first:first + N]
    hold = torch.full((3, 2 * M, N + 31), 7.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, ::2, first:first + N]
    run(g, out)
    assert rel(out, emulated(g)) <= U
    beside = hold.clone()
    beside[:, ::2, first:first + N] = 7.0
    assert torch.all(beside == 7.0)
    assert torch.equal(out, run(g.contiguous()))


def test_halves_of_gate_up():
    g = draw((2, 96, 2 * 144), torch.float32)
    out = torch.empty_like(g, dtype=torch.bfloat16)
    ws = moe.orthogonalize_workspace(g[:, :, :144])
    for i in (0, 1):
        run(g[:, :, 144 * i:144 * i + 144], out[:, :, 144 * i:144 * i + 144], ws)
    assert rel(out[:, :, :144], emulated(g[:, :, :144])) <= U and rel(out[:, :, 144:], emulated(g[:, :, 144:])) <= U


@pytest.mark.parametrize("M,N", [(100, 260), (260, 100), (300, 300)])
def test_in_place(M, N):
    g = draw((2, M, N), torch.bfloat16)
    want = run(g)
    run(g, g)
    assert torch.equal(g, want)


def test_broadcast_input():
    g = draw((48, 80), torch.float32)
    out = run(g.expand(3, 48, 80))
    assert torch.equal(out[0], run(g)) and torch.equal(out[1], out[0]) and torch.equal(out[2], out[0])


def test_repeats_bit_for_bit():
    for shape in ((5, 100, 700), (5, 500, 700), (2, 1500, 700)):
        g = draw(shape, torch.float32)
        want = run(g)
        assert all(torch.equal(run(g), want) for _ in range(3))


def test_two_streams_at_once():
    a, b, c = draw((4, 600, 900), torch.float32), draw((3, 700, 500), torch.bfloat16), draw((9, 60, 900), torch.float32)
    want = [run(t) for t in (a, b, c)]
    outs, wss = [torch.zeros_like(w) for w in want], [moe.orthogonalize_workspace(t) for t in (a, b, c)]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for t, o, ws, s in zip((a, b, c), outs, wss, streams):
            moe.orthogonalize(t, o, ws, stream=s)
    torch.cuda.synchronize()
    for ws in wss:
        moe.check_device_error(ws)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_steps_scale_and_coefficients():
    g = draw((2, 150, 280), torch.float32)
    for steps in (1, 2, 8):
        check(g, steps=steps)
    check(g, scale=-0.2)
    check(g, steps=6, coefs=[(1.5, -0.5, 0.0)] * 6)              # the cubic iteration
    per_step = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037),
                (2.8769, -3.1427, 1.2046), (2.8366, -3.0525, 1.2012)]
    check(g, coefs=per_step)
    assert torch.equal(run(g), run(g, coefs=COEFS))


def test_a_used_workspace_and_a_larger_one():
    g, other = draw((2, 150, 280), torch.float32), draw((3, 280, 300), torch.float32)
    want = run(g)
    ws = moe.orthogonalize_workspace(other)
    run(other, ws=ws)
    ws[256:].fill_(0xff)
    assert torch.equal(run(g, ws=ws), want)


def test_streams_and_graphs_on_one_workspace():
    a, b = draw((2, 150, 280), torch.float32), draw((2, 280, 150), torch.bfloat16)
    want = run(a), run(b)
    outs = [torch.zeros_like(w) for w in want]
    ws = moe.orthogonalize_workspace(a)
    graphs = []
    for g, o in zip((a, b), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.orthogonalize(g, o, ws)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    s = torch.cuda.Stream()
    outs[0].zero_()
    torch.cuda.synchronize()
    moe.orthogonalize(a, outs[0], ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0])


def test_empty_and_refused():
    e = torch.empty((0, 8, 8), device="cuda")
    moe.orthogonalize(e, e.to(torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"))
    g = draw((2, 16, 24), torch.float32)
    out, ws = torch.empty((2, 16, 24), dtype=torch.bfloat16, device="cuda"), moe.orthogonalize_workspace(g)
    for bad in (dict(steps=0), dict(steps=33), dict(eps=-1.0), dict(scale=float("inf")), dict(coefs=(1e6, 0.0, 0.0)),
                dict(coefs=(3.0, float("nan"), 0.0)), dict(coefs=(3.4445, -4.775, 9.0))):
        with pytest.raises(moe.MoeError):
            moe.orthogonalize(g, out, ws, **bad)
    for bad in ((g.mT, out.mT), (g, out.float()), (g, out[:1]), (g.double(), out), (g.cpu(), out), (g, out[0])):
        with pytest.raises(ValueError):
            moe.orthogonalize(bad[0], bad[1], ws)
    with pytest.raises(ValueError):
        moe.orthogonalize(g, out, ws, coefs=[COEFS] * 3)
    with pytest.raises(moe.MoeError):
        moe.orthogonalize(g, out, ws[:128])
    with pytest.raises(moe.MoeError):
        moe.orthogonalize(g, out[:1].expand(2, 16, 24), ws)        # results over one another


def test_a_wait_that_runs_out_is_reported():
    g = draw((2, 2048, 2048), torch.float32)     # waits long enough to be looked at
    want = run(g)
    ws, out = moe.orthogonalize_workspace(g), torch.empty_like(want)
    before = moe.moe_set_wait_timeout_ns(1)
    try:
        moe.orthogonalize(g, out, ws)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_timeout_ns(before)
    with pytest.raises(moe.MoeError):
        moe.check_device_error(ws)
    assert torch.equal(run(g, ws=ws), want)


def test_waits_without_a_limit():
    g = draw((2, 300, 300), torch.float32)
    want = run(g)
    before = moe.moe_set_wait_timeout_ns(2 ** 64 - 1)
    try:
        assert torch.equal(run(g), want)
    finally:
        moe.moe_set_wait_timeout_ns(before)


def roundings(g, steps=5, eps=1e-7):
    """The error in the 2-norm, relative to the result's, that the fp16 roundings leave.  A
    rounding has at most 2^-11 / sqrt(3) of its matrix's norm and points anywhere; those of
    x_j grow by c0 in every step to come, those of a and b reach x through the products (a
    random matrix times x has its norms' product over the root of m; a's by |c1| + 2 c2
    s^2) and grow by c0 from the next step on.  They are independent: the root of their
    squares' sum.  (c0 is the growth of what g does not contain, and more than that of
    what it does.)"""
    r = 2.0 ** -11 / math.sqrt(3)
    x = start(g, eps)
    x = x.mT if x.shape[-2] > x.shape[-1] else x
    m, t = x.shape[-2], 0.0
    c0, c1, c2 = COEFS
    for j in range(steps):
        a = x @ x.mT
        b = c0 * torch.eye(m, dtype=x.dtype, device=x.device) + c1 * a + c2 * (a @ a)
        n, s2 = float(x.norm()), float(torch.linalg.eigvalsh(a)[-1])
        to_come = c0 ** (steps - 1 - j)
        t += (r * n * c0 * to_come) ** 2
        t += (r * float(a.norm()) * n / math.sqrt(m) * (abs(c1) + 2 * c2 * s2) * to_come) ** 2
        t += (r * float(b.norm()) * n / math.sqrt(m) * to_come) ** 2
        x = b @ x
    return math.sqrt(t) / float(x.norm())


SPECTRA = {"falls to 1e-3": lambda k: 1e-3 ** (torch.arange(k) / (k - 1)), "falls to 1e-5": lambda k: 1e-5 ** (torch.arange(k) / (k - 1)),
           "as 1 / i": lambda k: 1.0 / torch.arange(1, k + 1), "half of the rank": lambda k: (torch.arange(k) < k // 2).float(),
           "rank 32": lambda k: (torch.arange(k) < 32).float(), "rank 4": lambda k: (torch.arange(k) < 4).float()}


@pytest.mark.parametrize("M,N", [(100, 700), (128, 64), (300, 140), (256, 512), (1030, 700)])
@pytest.mark.parametrize("name", list(SPECTRA))
def test_gradients_of_less_than_full_rank(M, N, name):
    """As of an expert with fewer tokens than rows, or singular values that fall off: the
    largest known case of what fp16 between the steps costs."""
    k = min(M, N)
    gen = torch.Generator().manual_seed(8)
    q = [torch.linalg.qr(torch.randn((n, k), generator=gen, dtype=torch.float64))[0] for n in (M, N)]
    g = ((q[0] * SPECTRA[name](k).double()) @ q[1].mT).float().cuda()
    err = rel(run(g), exact(g))
    assert err <= U + roundings(g)
    print("%s, %d x %d: %.1e of at most %.1e" % (name, M, N, err, U + roundings(g)))
