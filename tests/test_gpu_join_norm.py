"""A block's output joining the residual stream between two norms, and its gradient,
against the definitions in 64 bits.

Tolerances count roundings.  u is half a step of the type relative to the value
(finfo.eps / 2), u32 that of fp32.  An output is rounded once to its type (u).  Before
that, fp32 arithmetic: a row's sum (8 values a thread and vector, 5 + 5 steps of
butterflies: below 64 roundings), its root and quotient, and a handful of products:
below 96 u32 of the terms' magnitudes, which the bounds add up (a difference of terms
is off by the terms' errors, not by its own size).  The weights' gradients add the
rows in fp32: at most (rows per block + 64) further roundings."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
C = 96
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def half_step(dt):
    return torch.finfo(dt).eps / 2


def draw(shape, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt)


def cuda(t):
    return None if t is None else t.cuda()


class Case:
    def __init__(self, T, H, dt, post_norm=True, post_weight=True, gate=True, scale=1.0, seed=1, std=1.0):
        self.T, self.H, self.dt, self.post_norm, self.scale = T, H, dt, post_norm, scale
        self.y = draw((T, H), dt, seed, std)
        self.residual = draw((T, H), dt, seed + 1, 3 * std)
        self.wp = (1 + 0.1 * draw((H,), torch.float32, seed + 2)).to(dt) if post_weight else None
        self.w = (1 + 0.1 * draw((H,), torch.float32, seed + 3)).to(dt)
        self.gate = torch.sigmoid(draw((T,), torch.float32, seed + 4)) if gate else None

    def exact(self):
        y, r = self.y.double(), self.residual.double()
        rs_y = 1 / torch.sqrt(y.square().mean(-1) + EPS)
        p = y * rs_y[:, None] if self.post_norm else y
        if self.wp is not None:
            p = p * self.wp.double()
        if self.gate is not None:
            p = p * self.gate.double()[:, None]
        total = self.scale * r + p
        size = (self.scale * r).abs() + p.abs()          # the terms' magnitudes
        rs = 1 / torch.sqrt(total.square().mean(-1) + EPS)
        return rs_y, total, size, rs, total * rs[:, None] * self.w.double()

    def run(self, norm="same", total=None, n=None):
        T, H, dt = self.T, self.H, self.dt
        y, residual = self.y.cuda(), self.residual.cuda()
        out = {"total": torch.full((T, H), 7.0, dtype=dt, device="cuda") if total is None else {"y": y, "residual": residual}[total]}
        if self.post_norm:
            out["rs_y"] = torch.empty(T, device="cuda")
        if norm:
            out["rs"] = torch.empty(T, device="cuda")
            out["n"] = torch.empty((T, H), dtype=torch.uint8 if norm == "e4m3" else dt, device="cuda") if n is None else {"y": y, "residual": residual}[n]
        if norm == "e4m3":
            out["n_scale"] = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
        moe.join_norm_fwd(y, residual, out["total"], post_norm=self.post_norm, post_weight=cuda(self.wp),
                          gate=cuda(self.gate), residual_scale=self.scale, weight=cuda(self.w) if norm else None,
                          n=out.get("n"), n_scale=out.get("n_scale"), eps=EPS, rstd_post=out.get("rs_y"), rstd=out.get("rs"))
        return {k: v.cpu() for k, v in out.items()}

    def check(self, norm="same", **where):
        got = self.run(norm, **where)
        rs_y, total, size, rs, n = self.exact()
        u = half_step(self.dt)
        assert torch.all((got["total"].double() - total).abs() <= u * total.abs() + (1 + u) * C * U32 * size)
        if self.post_norm:
            assert torch.all((got["rs_y"].double() - rs_y).abs() <= 48 * U32 * rs_y)
        if not norm:
            return
        # the row's sum of squares: off by twice the terms' errors against its own size
        slack = 1 + 2 * (size * total.abs()).mean(-1) / (total.square().mean(-1) + EPS)
        assert torch.all((got["rs"].double() - rs).abs() <= C * U32 * slack * rs)
        nsize = size * rs[:, None] * self.w.double().abs()
        err = C * U32 * (nsize + slack[:, None] * n.abs())
        if norm == "same":
            assert torch.all((got["n"].double() - n).abs() <= u * n.abs() + (1 + u) * err + 1e-40)
            return
        b, e = n.view(self.T, -1, 32), err.view(self.T, -1, 32)
        amax, aerr = b.abs().amax(-1), e.amax(-1)
        scale = torch.exp2(got["n_scale"].double() - 127)
        live = amax > 0
        # the smallest power of two with amax <= 448 scale, up to amax's error
        assert torch.all((448 * scale >= amax - aerr)[live]) and torch.all((224 * scale <= amax + aerr)[live])
        code = got["n"].view(torch.float8_e4m3fn).double().view(self.T, -1, 32)
        v, e = b / scale[..., None], e / scale[..., None]
        # half a step of e4m3 (2^-4 of the value's power of two, at least half of 2^-9),
        # at 448 one more where the error passes it
        step = torch.exp2(torch.floor(torch.log2((v.abs() + e).clamp(min=2.0 ** -6))) - 3)
        assert torch.all((code - v).abs() <= 0.5 * step + e)


SIZES = [(1, 8), (1, 2880), (3, 32), (5, 2880), (7, 4096), (33, 264), (2, 8192), (2, 8200), (3, 16384), (2, 32768), (513, 128)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward(T, H, dtype):
    Case(T, H, DT[dtype]).check()
    Case(T, H, DT[dtype], post_weight=False, gate=False, scale=0.5).check()
    Case(T, H, DT[dtype], post_norm=False, gate=False, scale=1.5).check()
    Case(T, H, DT[dtype], post_norm=False, post_weight=False).check("")
    Case(T, H, DT[dtype]).check("")


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2880), (5, 4096), (9, 96), (2, 8192), (2, 16384), (2, 32768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_8bit(T, H, dtype):
    Case(T, H, DT[dtype]).check("e4m3")
    Case(T, H, DT[dtype], post_norm=False, scale=-0.5).check("e4m3")


@pytest.mark.parametrize("T,H", [(1400, 288), (1300, 2912), (700, 5152), (640, 8224), (330, 16416)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", ["same", "e4m3", ""])
def test_forward_several_rows_per_block(T, H, dtype, norm):
    """More rows than resident blocks, and warps that a row's end cuts."""
    Case(T, H, DT[dtype]).check(norm)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("total,n", [("y", None), ("residual", None), (None, "y"), (None, "residual"), ("y", "residual"), ("residual", "y")])
@pytest.mark.parametrize("T", [5, 1400])
def test_outputs_over_inputs(T, dtype, total, n):
    Case(T, 264, DT[dtype]).check(total=total, n=n)


def test_sum_that_cancels():
    """The residual is nearly what joins it: the sum of squares of what is left, not of
    the terms, sets the next norm."""
    c = Case(6, 256, torch.float32, post_weight=False, gate=False)
    y = c.y.double()
    c.residual = (-y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) + 1e-3 * draw((6, 256), torch.float64, 9)).float()
    c.check()
    c.check("e4m3")


def test_scales_and_zero_rows():
    Case(4, 256, torch.float32, std=1e-12).check()
    Case(4, 256, torch.float32, std=1e15).check()
    c = Case(4, 256, torch.bfloat16)
    c.y[1] = 0
    c.y[2], c.residual[2] = 0, 0
    c.gate[3] = 0
    c.check()
    c.check("e4m3")
    assert c.run("e4m3")["n_scale"][2].tolist() == [0] * 8


def test_non_finite_rows_stay_apart():
    c = Case(4, 64, torch.bfloat16)
    c.y[1, 3] = float("nan")
    c.residual[2, 40] = float("inf")
    got = c.run()
    assert torch.isnan(got["total"][1]).all() and torch.isnan(got["n"][1]).all()
    assert torch.isinf(got["total"][2, 40]) and torch.isnan(got["n"][2, 40])
    assert torch.isfinite(got["total"][[0, 3]]).all() and torch.isfinite(got["n"][[0, 3]]).all()
    assert torch.isfinite(got["total"][2, :40]).all() and torch.all(got["n"][2, :40] == 0)


class Grad(Case):
    def __init__(self, T, H, dt, next_norm=True, d_total=True, seed=21, **kw):
        super().__init__(T, H, dt, seed=seed, **kw)
        rs_y, total, _, rs, _ = self.exact()
        self.total, self.rs_y, self.rs = total.to(dt), rs_y.float(), rs.float()
        self.dn = draw((T, H), dt, seed + 6) if next_norm else None
        self.d_total = draw((T, H), dt, seed + 7) if d_total else None

    def grads(self):
        """({name: (value, bound before the output's rounding)}, by the formulas in 64 bits."""
        one = torch.ones((), dtype=torch.float64)
        gate = self.gate.double()[:, None] if self.gate is not None else one
        wp = self.wp.double() if self.wp is not None else one
        rs_y = self.rs_y.double()[:, None] if self.post_norm else one
        yhat = self.y.double() * rs_y
        dr = self.d_total.double() if self.d_total is not None else torch.zeros((self.T, self.H), dtype=torch.float64)
        size = dr.abs()
        out = {}
        if self.dn is not None:
            rs, rhat = self.rs.double()[:, None], self.total.double() * self.rs.double()[:, None]
            v = self.dn.double() * self.w.double()
            dr = dr + rs * (v - rhat * (v * rhat).mean(-1, keepdim=True))
            size = size + rs * (v.abs() + rhat.abs() * (v * rhat).abs().mean(-1, keepdim=True))
            t = self.dn.double() * rhat
            out["d_weight"] = (t.sum(0), (C + self.T) * U32 * t.abs().sum(0))
        q = yhat * wp
        D, Dsize = (dr * q).sum(-1, keepdim=True), (size * q.abs()).sum(-1, keepdim=True)
        out["d_gate"] = (D[:, 0], 2 * C * U32 * Dsize[:, 0])
        dy = gate * dr * wp
        dysize = gate * size * wp.abs()
        if self.post_norm:
            dy = rs_y * (dy - yhat * gate * D / self.H)
            dysize = rs_y * (dysize + 2 * yhat.abs() * gate * Dsize / self.H)
        out["dy"] = (dy, C * U32 * dysize)
        out["d_residual"] = (self.scale * dr, C * U32 * abs(self.scale) * size)
        out["d_post_weight"] = ((gate * dr * yhat).sum(0), (2 * C + self.T) * U32 * (gate * size * yhat.abs()).sum(0))
        return out

    def run_bwd(self, dy=None, d_residual=None, sums=True):
        T, H = self.T, self.H
        t = {n: cuda(getattr(self, n)) for n in ("y", "d_total", "dn", "total")}
        if self.dn is None:
            t["total"] = None
        out = {"dy": torch.empty((T, H), dtype=self.dt, device="cuda") if dy is None else t[dy],
               "d_residual": torch.empty((T, H), dtype=self.dt, device="cuda") if d_residual is None else t[d_residual],
               "d_gate": torch.empty(T, device="cuda")}
        if sums:
            out["d_post_weight"] = torch.full((H,), 3.0, device="cuda")
            if self.dn is not None:
                out["d_weight"] = torch.full((H,), 3.0, device="cuda")
        moe.join_norm_bwd(t["y"], out["dy"], out["d_residual"], d_total=t["d_total"], dn=t["dn"], total=t["total"],
                          weight=cuda(self.w) if self.dn is not None else None, rstd=cuda(self.rs) if self.dn is not None else None,
                          post_norm=self.post_norm, post_weight=cuda(self.wp), rstd_post=cuda(self.rs_y) if self.post_norm else None,
                          gate=cuda(self.gate), residual_scale=self.scale, d_gate=out["d_gate"],
                          d_post_weight=out.get("d_post_weight"), d_weight=out.get("d_weight"),
                          ws=moe.join_norm_workspace(T, H) if sums else None)
        return {k: v.cpu() for k, v in out.items()}

    def check_bwd(self, **where):
        got, want = self.run_bwd(**where), self.grads()
        u = half_step(self.dt)
        for name, v in got.items():
            ref, err = want[name]
            once = u if name in ("dy", "d_residual") else U32
            assert torch.all((v.double() - ref).abs() <= once * ref.abs() + (1 + once) * err + 1e-40), name
        return got


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2880), (3, 32), (700, 2880), (65, 4096), (33, 264), (5, 8200), (3, 16384), (2, 32768), (2049, 128), (400, 8208)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward(T, H, dtype):
    Grad(T, H, DT[dtype]).check_bwd()
    Grad(T, H, DT[dtype], next_norm=False, scale=0.5).check_bwd()
    Grad(T, H, DT[dtype], d_total=False, post_weight=False, gate=False).check_bwd()
    Grad(T, H, DT[dtype], post_norm=False, scale=1.5).check_bwd()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dy,d_residual", [("dn", "d_total"), ("y", "total"), ("total", "y"), ("d_total", "dn")])
@pytest.mark.parametrize("T", [5, 1400])
def test_backward_over_inputs(T, dtype, dy, d_residual):
    Grad(T, 264, DT[dtype]).check_bwd(dy=dy, d_residual=d_residual)


@pytest.mark.parametrize("T,H", [(1, 8208), (150, 9000), (320, 8712), (230, 16384), (90, 16392), (161, 32768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_of_wide_rows(T, H, dtype):
    """Rows on several CTAs, one row and several for each."""
    Grad(T, H, DT[dtype]).check_bwd()
    Grad(T, H, DT[dtype], next_norm=False, post_norm=False, gate=False).check_bwd()
    c = Grad(T, H, DT[dtype], d_total=False, scale=0.5)
    a, b = c.check_bwd(), c.run_bwd()
    assert all(torch.equal(a[k], b[k]) for k in a)
    a = c.run_bwd(dy="dn", d_residual="y")
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_backward_without_weight_gradients():
    Grad(700, 2880, torch.bfloat16).check_bwd(sums=False)


def test_backward_repeats_bit_for_bit():
    c = Grad(3000, 520, torch.bfloat16)
    a, b = c.run_bwd(), c.run_bwd()
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradient_against_differences():
    """The forward's own differences: a quotient over 2 h of fp32 results that carry
    C u32 of their size each, plus h^2 for the third derivative (values of order 1)."""
    T, H = 3, 64
    c = Grad(T, H, torch.float32, scale=0.7)
    c.total = c.exact()[1].float()
    got = c.run_bwd()
    g = torch.Generator().manual_seed(5)

    def loss(**change):
        keep = {k: getattr(c, k) for k in change}
        for k, v in change.items():
            setattr(c, k, v)
        out = c.run()
        for k, v in keep.items():
            setattr(c, k, v)
        return float((out["total"].double() * c.d_total.double()).sum() + (out["n"].double() * c.dn.double()).sum())

    h = 2.0 ** -6
    size = float((c.exact()[2].abs() * c.d_total.double().abs()).sum() + (c.exact()[4].abs() * c.dn.double().abs()).sum())
    for name, grad in (("y", got["dy"]), ("residual", got["d_residual"]), ("gate", got["d_gate"]),
                       ("wp", got["d_post_weight"]), ("w", got["d_weight"])):
        x = getattr(c, name)
        d = torch.randn(x.shape, generator=g)
        d /= d.norm()
        slope = (loss(**{name: x + h * d}) - loss(**{name: x - h * d})) / (2 * h)
        want = float((grad.double() * d.double()).sum())
        assert abs(slope - want) <= C * U32 * size / h + 20 * h * h * float(grad.double().norm()), name


def test_empty_and_refused():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    moe.join_norm_fwd(e, e, e)
    f = torch.empty(0, device="cuda")
    moe.join_norm_fwd(e, e, e, gate=f, weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"), n=e, rstd_post=f, rstd=f)
    dw, dwp = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    moe.join_norm_bwd(e, e, e, d_total=e, post_norm=False, d_post_weight=dwp)
    assert not dwp.any()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    moe.join_norm_bwd(e, e, e, dn=e, total=e, weight=w, rstd=torch.empty(0, device="cuda"), post_norm=False, d_weight=dw)
    assert not dw.any()
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(x)
    with pytest.raises(moe.MoeError):
        moe.join_norm_fwd(x, x, o, weight=w, n=o)                  # total and n the same
    with pytest.raises(moe.MoeError):
        moe.join_norm_bwd(x, o, o, d_total=x, post_norm=False)     # dy and d_residual the same
    with pytest.raises(ValueError):
        moe.join_norm_bwd(x, x, o, d_total=x)                      # a post norm without its 1 / rms
    with pytest.raises(ValueError):
        moe.join_norm_fwd(x, x[:, ::2], o)
    with pytest.raises(ValueError):
        moe.join_norm_fwd(x, x.float(), o)
    with pytest.raises(moe.MoeError):
        moe.join_norm_bwd(x, o, torch.empty_like(x), d_total=x, post_norm=False, d_post_weight=dw)   # no workspace


def test_other_stream_and_graph():
    c = Grad(700, 264, torch.bfloat16)
    want = c.run_bwd()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t = {n: getattr(c, n).cuda() for n in ("y", "d_total", "dn", "total", "w", "wp", "gate", "rs", "rs_y")}
    out = [torch.zeros((700, 264), dtype=c.dt, device="cuda") for _ in range(2)]
    sums = [torch.zeros(264, device="cuda") for _ in range(2)]
    ws = moe.join_norm_workspace(700, 264)
    torch.cuda.synchronize()

    def go(stream=None):
        moe.join_norm_bwd(t["y"], *out, d_total=t["d_total"], dn=t["dn"], total=t["total"], weight=t["w"], rstd=t["rs"],
                          post_weight=t["wp"], rstd_post=t["rs_y"], gate=t["gate"], d_post_weight=sums[0], d_weight=sums[1],
                          ws=ws, stream=stream)

    def same():
        torch.cuda.synchronize()
        return (torch.equal(out[0].cpu(), want["dy"]) and torch.equal(out[1].cpu(), want["d_residual"])
                and torch.equal(sums[0].cpu(), want["d_post_weight"]) and torch.equal(sums[1].cpu(), want["d_weight"]))

    go(s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for o in out + sums:
        o.zero_()
    ws.fill_(0xff)                 # what the workspace holds does not matter
    graph.replay()
    graph.replay()
    assert same()
