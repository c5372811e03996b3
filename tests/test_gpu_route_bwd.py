"""The router's gradient (chosen weights, load-balancing loss, z-loss) against the
definitions in 64 bits.

Tolerances: an exponential's argument v - max carries |v - max| u32, so a probability
is off by that and a handful of roundings relative to itself; sums over a row below 48
roundings.  The bound adds the terms' magnitudes with (64 + |v - max|) u32."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2


class Case:
    def __init__(self, T, E, k, balance=0.02, z=0.001, weights=True, seed=1, std=2.0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.E, self.k, self.balance, self.z = T, E, k, balance, z
        self.logits = torch.randn((T, E), generator=g) * std
        top = torch.topk(self.logits, k, dim=-1)
        self.idx, self.w = top.indices.to(torch.int32), torch.softmax(top.values, dim=-1)
        self.counts = torch.bincount(self.idx.flatten().long(), minlength=E).to(torch.int32)
        self.dw = torch.randn((T, k), generator=g) * 0.1 if weights else None

    def exact(self):
        v = self.logits.double()
        top = v.amax(-1, keepdim=True)
        alive = torch.isfinite(top)
        p = torch.where(alive, torch.softmax(v, -1), torch.zeros_like(v))
        lse = torch.where(alive, torch.logsumexp(v, -1, keepdim=True), torch.zeros_like(top))
        f = self.counts.double() * self.E / (self.T * self.k)
        F = (f * p).sum(-1, keepdim=True)
        a, b = self.balance / self.T, 2 * self.z / self.T
        d = a * p * (f - F) + b * lse * p
        reach = torch.where(p > 0, (v - top).abs(), torch.zeros_like(v))
        size = (a * p * (f + F) + b * (lse.abs() + top.nan_to_num(0, 0, 0).abs()) * p) * (64 + reach)
        if self.dw is not None:
            w, dw = self.w.double(), self.dw.double()
            ok = (self.idx >= 0) & (self.idx < self.E)
            c = w * (dw - (w * dw).sum(-1, keepdim=True))
            at = self.idx.long().clamp(0, self.E - 1)
            d.scatter_add_(1, at, c * ok)
            size.scatter_add_(1, at, 64 * w * (dw.abs() + (w * dw).abs().sum(-1, keepdim=True)) * ok)
        return d, U32 * size, torch.stack((F.mean(), lse.square().mean()))

    def run(self, losses=True, stream=None, counts=True, logits=True):
        shape = moe.Shape(self.T, 8, 8, self.E, self.k)
        ws = moe.route_bwd_workspace(shape)
        d = torch.full((self.T, self.E), 7.0, device="cuda")
        out = torch.full((2,), 7.0, device="cuda") if losses else None
        moe.route_bwd(shape, self.logits.cuda() if logits else None, d, ws, topk_idx=self.idx.cuda(), topk_w=self.w.cuda(),
                      d_topk_w=None if self.dw is None else self.dw.cuda(), counts=self.counts.cuda() if counts else None,
                      balance=self.balance, z=self.z, losses=out)
        torch.cuda.synchronize()
        return d.cpu(), None if out is None else out.cpu(), ws

    def check(self, **kw):
        d, losses, ws = self.run(**kw)
        ref, bound, ref_losses = self.exact()
        assert torch.all((d.double() - ref).abs() <= U32 * ref.abs() + bound + 1e-44)
        if losses is not None:
            # F and the square of log sum exp: below 64 + |v| roundings each, all of one
            # sign; a loss beyond fp32's range (logits past 1e19) rounds to infinity
            far = torch.isinf(ref_losses.float())
            assert torch.all(torch.isposinf(losses[far]))
            losses, ref_losses = losses[~far], ref_losses[~far]
            assert torch.all((losses.double() - ref_losses).abs() <= (80 + 2 * float(self.logits.nan_to_num(0, 0, 0).abs().max())) * U32 * ref_losses + 1e-44)
        return ws


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 4), (3, 5, 2), (37, 61, 6), (8, 128, 4), (1000, 128, 4), (5, 129, 8), (64, 256, 8),
                                   (33, 255, 3), (9, 512, 8), (6, 511, 32), (4, 1024, 32), (7, 1023, 8), (20000, 32, 2), (12000, 60, 5), (2, 40, 32)])
def test_gradient(T, E, k):
    Case(T, E, k).check()
    Case(T, E, k, weights=False).check()
    Case(T, E, k, balance=0.0, z=0.0).check()
    Case(T, E, k, balance=0.0, z=0.0).check(losses=False, counts=False, logits=False)
    Case(T, E, k, balance=0.5, z=0.0).check(losses=False)


def test_against_differences():
    """Of the losses and the weights that the framework's own forward gives."""
    c = Case(6, 24, 3, std=1.0)
    d, _, _ = c.run()
    g = torch.Generator().manual_seed(9)
    direction = torch.randn(c.logits.shape, generator=g, dtype=torch.float64)
    direction /= direction.norm()

    def loss(v):
        chosen = torch.softmax(v.gather(1, c.idx.long()), -1)
        f = c.counts.double() * c.E / (c.T * c.k)
        return float((chosen * c.dw.double()).sum() + c.balance * (torch.softmax(v, -1).mean(0) * f).sum()
                     + c.z * torch.logsumexp(v, -1).square().mean())

    h = 2.0 ** -12
    slope = (loss(c.logits.double() + h * direction) - loss(c.logits.double() - h * direction)) / (2 * h)
    assert abs(slope - float((d.double() * direction).sum())) <= 64 * U32 * float(d.double().norm()) + h * h


def test_masked_experts_and_rows():
    c = Case(6, 40, 4)
    c.logits[:, 7] = float("-inf")
    c.logits[2, 3:] = float("-inf")
    c.logits[4] = float("-inf")
    c.logits[5] = -3.0e38
    c.idx[:, :] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    c.check()
    c.dw = None
    d, _, _ = c.run()
    assert torch.isfinite(d).all() and not d[4].any() and not d[:5, 7].any()      # (row 5 masks none)


def test_non_finite_rows_stay_apart():
    c = Case(5, 40, 4)
    c.logits[1, 5] = float("nan")
    c.logits[3, 5] = float("inf")
    d, losses, _ = c.run()
    assert torch.isnan(d[1]).all() and torch.isnan(losses).all()
    assert torch.isfinite(d[[0, 2, 4]]).all()


def test_large_logits():
    Case(9, 100, 4, std=1e4).check()
    Case(9, 100, 4, std=1e-20).check()


def test_the_same_expert_twice():
    c = Case(5, 128, 6)
    c.idx[1] = 3
    c.idx[2, :2] = c.idx[2, 2]
    c.check()
    c = Case(5, 33, 32)
    c.idx[0] = 32
    c.check()


def test_bad_ids_are_reported_and_add_nothing():
    c = Case(5, 128, 4)
    c.idx[1, 2], c.idx[3, 0] = 128, -1
    ws = c.check()
    with pytest.raises(moe.MoeError):
        moe.check_device_error(ws)
    moe.check_device_error(ws)        # read and cleared


def test_no_rows():
    shape = moe.Shape(0, 8, 8, 16, 2)
    losses = torch.full((2,), 7.0, device="cuda")
    moe.route_bwd(shape, torch.empty((0, 16), device="cuda"), torch.empty((0, 16), device="cuda"),
                  moe.route_bwd_workspace(shape), balance=1.0, counts=torch.zeros(16, dtype=torch.int32, device="cuda"), losses=losses)
    assert not losses.any()


def test_repeats_bit_for_bit_and_in_a_graph():
    c = Case(5000, 100, 4)
    d0, l0, _ = c.run()
    shape = moe.Shape(c.T, 8, 8, c.E, c.k)
    t = [v.cuda() for v in (c.logits, c.idx, c.w, c.dw, c.counts)]
    ws, d, losses = moe.route_bwd_workspace(shape), torch.zeros((c.T, c.E), device="cuda"), torch.zeros(2, device="cuda")

    def go(stream=None):
        moe.route_bwd(shape, t[0], d, ws, t[1], t[2], t[3], t[4], c.balance, c.z, losses, stream)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    go(s)
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), d0) and torch.equal(losses.cpu(), l0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    d.zero_(), losses.zero_()
    ws[256:].fill_(0xff)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), d0) and torch.equal(losses.cpu(), l0)


def test_sizes_in_turn_on_one_workspace():
    """Calls of one block, of one round of many and of several rounds: each leaves the
    workspace as the others want it."""
    ws, cases, want = moe.route_bwd_workspace(moe.Shape(20000, 8, 8, 64, 4)), [], []
    for T in (5, 20000, 700, 33, 2000, 20000, 64, 1):
        shape = moe.Shape(T, 8, 8, 64, 4)
        logits = torch.randn((T, 64), generator=torch.Generator().manual_seed(T)).cuda()
        counts = torch.full((64,), T // 16 + 1, dtype=torch.int32, device="cuda")
        args = (shape, logits, counts, torch.zeros_like(logits), torch.zeros(2, device="cuda"))
        cases.append(args)
        fresh = [torch.zeros_like(logits), torch.zeros(2, device="cuda")]
        moe.route_bwd(shape, logits, fresh[0], moe.route_bwd_workspace(shape), counts=counts, balance=0.1, z=0.1, losses=fresh[1])
        p = torch.softmax(logits.double(), -1)
        f = counts.double() * 64 / (T * 4)
        exact = torch.stack(((p @ f).mean(), torch.logsumexp(logits.double(), -1).square().mean()))
        # sums of positive terms, at most some 40 fp32 additions deep
        assert torch.all((fresh[1].double() - exact).abs() <= 64 * 2.0 ** -24 * exact)
        want.append(fresh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for shape, logits, counts, d, losses in cases:
            moe.route_bwd(shape, logits, d, ws, counts=counts, balance=0.1, z=0.1, losses=losses)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for (_, _, _, d, losses), (wd, wl) in zip(cases, want):
            assert torch.equal(d, wd) and torch.equal(losses, wl)
            d.zero_(), losses.zero_()


def test_refusals():
    c = Case(4, 16, 2)
    shape = moe.Shape(4, 8, 8, 16, 2)
    ws, d = moe.route_bwd_workspace(shape), torch.empty((4, 16), device="cuda")
    v, idx, w, dw, counts = [t.cuda() for t in (c.logits, c.idx, c.w, c.dw, c.counts)]
    for bad in (dict(counts=None, balance=1.0), dict(topk_idx=None), dict(topk_w=None), dict(z=float("inf"))):
        args = dict(topk_idx=idx, topk_w=w, d_topk_w=dw, counts=counts)
        args.update(bad)
        with pytest.raises(moe.MoeError):
            moe.route_bwd(shape, v, d, ws, **args)
    with pytest.raises(ValueError):
        moe.route_bwd(shape, v[:, :8], d, ws, z=1.0, counts=counts)
    with pytest.raises(ValueError):
        moe.route_bwd(shape, v, d, ws, topk_idx=idx.long(), topk_w=w, d_topk_w=dw)
    with pytest.raises(moe.MoeError):
        moe.route_bwd(shape, v, d, ws[:256], z=1.0, counts=counts)


@pytest.mark.parametrize("fill", [0x01, 0xA5, 0xFF])
@pytest.mark.parametrize("T,E,k", [(1000, 128, 4), (5000, 61, 4), (70, 256, 8)])
def test_only_the_error_word_is_kept_in_the_workspace(T, E, k, fill):
    """Whatever the rest of the workspace holds, its header too."""
    c = Case(T, E, k)
    shape = moe.Shape(T, 8, 8, E, k)
    ws = moe.route_bwd_workspace(shape)
    d0, l0, _ = c.run()
    t = [v.cuda() for v in (c.logits, c.idx, c.w, c.dw, c.counts)]
    for _ in range(3):
        ws[4:].fill_(fill)
        d, losses = torch.zeros((T, E), device="cuda"), torch.zeros(2, device="cuda")
        moe.route_bwd(shape, t[0], d, ws, t[1], t[2], t[3], t[4], c.balance, c.z, losses)
        assert torch.equal(d.cpu(), d0) and torch.equal(losses.cpu(), l0)
    moe.check_device_error(ws)


@pytest.mark.parametrize("E", [60, 128, 255, 500, 1024])
def test_probabilities_to_fp32s_roundings(E):
    """The error's 2-norm, against roundings that are as likely to go either way (each u32 /
    sqrt(3) at most): the balance loss's gradient p_e (f_e - F) where one expert alone has
    tokens, so nothing cancels but in its column, left out here.  The logits' differences
    are exact.  An exponential and a quotient to 2 ulp each (4 u32 / sqrt(3) = 2.3 u32), a
    row's sum at most 32 + 5 additions deep but adding the small to the large (2.1 u32 as
    for 13 of equal size), sum and quotient twice (6.2 u32), the sum of F and eight further
    roundings: 7.1 u32 in all."""
    c = Case(600, E, 2, balance=1.0, z=0.0, weights=False)
    c.logits = (c.logits * 64).round() / 64
    c.counts.zero_()
    c.counts[E // 3] = 77
    d, _, _ = c.run(losses=False)
    want = c.exact()[0]
    keep = torch.arange(E) != E // 3
    err = (d.double() - want)[:, keep].norm() / want[:, keep].norm()
    assert err <= 8 * U32


def test_probabilities_far_below_the_largest():
    """Down to the least fp32 number: 2 ulp of the exponential and what a subnormal's place
    rounds (half of 2^-149, times the factors behind it)."""
    c = Case(1, 200, 2, balance=1.0, z=0.0, weights=False)
    c.logits[0] = -torch.arange(200) * 0.53125
    c.counts.zero_()
    c.counts[0] = 2
    d, _, _ = c.run(losses=False)
    want = c.exact()[0]
    assert d[0, 1:].min() < 0 and d[0, 150] != 0
    # |d| = p f_0 p_0 with f_0 = E / 2 * 2 / k = 100 here: a subnormal p's half step by 100
    assert torch.all((d.double() - want).abs()[0, 1:] <= 64 * U32 * want.abs()[0, 1:] + 200 * 2.0 ** -150)


@pytest.mark.parametrize("T,E,k", [(100000, 32, 2), (100001, 62, 6), (50000, 128, 16), (50001, 127, 16), (25000, 256, 8), (25001, 255, 8),
                                   (20000, 512, 8), (20001, 511, 8), (7000, 1024, 32), (7001, 1023, 32)])
def test_many_rows_per_warp(T, E, k):
    """At least five rows for each, so that all stages of the copies ahead are used again,
    and a last round that not all warps have."""
    Case(T, E, k).check()
    Case(T, E, k, weights=False, balance=0.3, z=0.0).check()
    Case(T, E, k, balance=0.0, z=0.0).check(losses=False, counts=False, logits=False)
