"""Host-side checks of a training step's operators: what their C entry points refuse
before any device access, and their workspace sizes."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from dispatch_gemm_combine_gb300 import _build
    _build.build()
    import dispatch_gemm_combine_gb300 as m
    return m


def test_join_norm_refusals(L):
    ok = dict(T=4, H=64, dtype=L.MOE_BF16, y=16, residual=16, post_norm=1, post_weight=16, gate=4, residual_scale=1.0,
              weight=16, eps=1e-6, total=32, n=48, n_scale=None, rstd_post=4, rstd=4, stream=None)
    bad = [dict(H=12), dict(H=0), dict(H=40000), dict(T=-1), dict(T=1 << 31), dict(dtype=7), dict(y=None),
           dict(residual=None), dict(total=None), dict(y=8), dict(residual=8), dict(post_weight=8), dict(weight=8),
           dict(total=8), dict(n=8), dict(n=None), dict(weight=None), dict(n=32), dict(eps=-1.0), dict(eps=float("nan")),
           dict(residual_scale=float("nan")), dict(residual_scale=float("inf")), dict(post_norm=2), dict(post_norm=0),
           dict(H=40, n_scale=16), dict(weight=None, n=None, n_scale=16), dict(weight=None, n=None)]
    for b in bad:
        assert L.moe_join_norm_fwd(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    assert L.moe_join_norm_fwd(**dict(ok, T=0, y=None, residual=None, total=None)) == L.MOE_OK

    ok = dict(T=4, H=64, dtype=L.MOE_BF16, dn=16, d_total=16, total=16, rstd=4, weight=16, y=16, rstd_post=4,
              post_weight=16, gate=4, residual_scale=1.0, dy=32, d_residual=48, d_gate=4, d_post_weight=16, d_weight=16,
              ws=256, ws_bytes=1 << 30, stream=None)
    bad = [dict(H=12), dict(T=-1), dict(dtype=2), dict(y=None), dict(dy=None), dict(d_residual=None), dict(dy=48),
           dict(dn=None, d_total=None), dict(total=None), dict(rstd=None), dict(weight=None), dict(dn=None), dict(dn=8),
           dict(d_total=8), dict(total=8), dict(weight=8), dict(y=8), dict(post_weight=8), dict(dy=8), dict(d_residual=8),
           dict(d_post_weight=8), dict(d_weight=8), dict(ws=None), dict(ws=16), dict(residual_scale=float("nan"))]
    for b in bad:
        assert L.moe_join_norm_bwd(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    need = L.moe_join_norm_workspace_size(4, 64)
    assert need >= 2 * 4 * 64 * 4
    assert L.moe_join_norm_bwd(**dict(ok, ws_bytes=need - 1)) == L.MOE_ERR_WORKSPACE
    assert L.moe_join_norm_workspace_size(4, 65) == 0 and L.moe_join_norm_workspace_size(-1, 64) == 0


def test_route_bwd_refusals(L):
    s = L.Shape(4, 8, 8, 16, 2)
    size = L.moe_route_bwd_workspace_size(s)
    assert size > 256 and L.moe_route_bwd_workspace_size(L.Shape(4, 8, 8, 16, 17)) == 0
    ok = dict(shape=s, logits=16, topk_idx=4, topk_w=4, counts=4, d_topk_w=4, balance=0.1, z=0.1, d_logits=32, losses=4,
              ws=256, ws_bytes=size, stream=None)
    for b in (dict(shape=L.Shape(-1, 8, 8, 16, 2)), dict(shape=L.Shape(4, 8, 8, 2000, 2)), dict(logits=None), dict(counts=None),
              dict(topk_idx=None), dict(topk_w=None), dict(d_logits=None), dict(ws=None), dict(ws=128), dict(logits=8),
              dict(d_logits=8), dict(balance=float("nan")), dict(z=float("inf"))):
        assert L.moe_route_bwd(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    assert L.moe_route_bwd(**dict(ok, ws_bytes=size - 1)) == L.MOE_ERR_WORKSPACE


def test_orthogonalize_refusals(L):
    size = L.moe_orthogonalize_workspace_size(2, 16, 24)
    assert size >= 256
    # two copies of x, a and b in fp16
    assert L.moe_orthogonalize_workspace_size(2, 300, 500) >= 2 * 2 * 300 * (500 + 500 + 300 + 300)
    for bad in ((-1, 16, 24), (2, 0, 24), (2, 16, 0), (2, 65537, 4), (2, 4, 65537)):
        assert L.moe_orthogonalize_workspace_size(*bad) == 0
    # the workspace is that of the matrices that go through at once
    assert L.moe_orthogonalize_workspace_size(4096, 2880, 2880) == L.moe_orthogonalize_workspace_size(64, 2880, 2880)
    for M, N in ((129, 65536), (2880, 5760), (140, 300)):
        assert L.moe_orthogonalize_workspace_size(1 << 30, M, N) < (5 << 28)
    # that of the transposes, and no less for more matrices
    for M, N in ((300, 5000), (2880, 2880), (129, 40000), (1000, 1200), (64, 9000)):
        sizes = [L.moe_orthogonalize_workspace_size(E, M, N) for E in (0, 1, 2, 3, 7, 40, 1000)]
        assert sizes == [L.moe_orthogonalize_workspace_size(E, N, M) for E in (0, 1, 2, 3, 7, 40, 1000)]
        assert sizes == sorted(sizes)
    ok = dict(E=2, M=16, N=24, dtype=L.MOE_FP32, g=16, g_ld=24, g_stride=384, steps=5, coefs=None, eps=1e-7, scale=1.0,
              out=16, out_ld=24, out_stride=384, ws=256, ws_bytes=size, stream=None)

    def coefs(*v):
        return (ctypes.c_float * len(v))(*v)

    for b in (dict(E=-1), dict(M=0), dict(N=65537), dict(dtype=3), dict(g=None), dict(out=None), dict(g=18), dict(out=17),
              dict(g_ld=23), dict(out_ld=23), dict(g_stride=-1), dict(out_stride=383), dict(out_stride=0), dict(steps=0),
              dict(steps=33), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("nan")),
              dict(ws=None), dict(ws=128), dict(coefs=coefs(*[1e5, 0.0, 0.0] * 5)), dict(coefs=coefs(*[3.0, float("nan"), 0.0] * 5)),
              dict(coefs=coefs(*[3.4445, -4.775, 2.0315] * 4, 3.0, float("inf"), 0.0))):
        assert L.moe_orthogonalize(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    assert L.moe_orthogonalize(**dict(ok, ws_bytes=size - 1)) == L.MOE_ERR_WORKSPACE
    assert L.moe_orthogonalize(**dict(ok, E=0, g=None, out=None, ws=None, ws_bytes=0)) == L.MOE_OK


def test_orthogonalize_refuses_scales_that_fp32_loses(L):
    size = L.moe_orthogonalize_workspace_size(2, 16, 24)
    ok = dict(E=2, M=16, N=24, dtype=L.MOE_FP32, g=16, g_ld=24, g_stride=384, steps=5, coefs=None, eps=1e-7, scale=1.0,
              out=16, out_ld=24, out_stride=384, ws=256, ws_bytes=size, stream=None)
    for scale in (1e-38, -1e-38, 2.0 ** -101, 1e-45):
        assert L.moe_orthogonalize(**dict(ok, scale=scale)) == L.MOE_ERR_INVALID_ARG
    # (E = 0: nothing is launched)
    for scale in (0.0, 2.0 ** -100, -1.0):
        assert L.moe_orthogonalize(**dict(ok, E=0, scale=scale)) == L.MOE_OK


def test_helpers_refuse_coefficients(L):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for coefs, steps in (([], 0), ([], 5), ((1.0, 2.0), 5), ([(1.0, 2.0, 3.0)], 2), ((1.0, 2.0, 3.0), 10 ** 9), ((1.0, 2.0, 3.0), -1)):
        with pytest.raises(ValueError, match="coefficients"):
            L.orthogonalize(x, x, torch.zeros(8, dtype=torch.uint8), steps=steps, coefs=coefs)


def test_helpers_refuse_tensors_on_the_host(L):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.join_norm_fwd(x, x, x)
    with pytest.raises(ValueError):
        L.join_norm_bwd(x, x, x, d_total=x, post_norm=False)
    with pytest.raises(ValueError):
        L.route_bwd(L.Shape(4, 8, 8, 16, 2), torch.zeros((4, 16)), torch.zeros((4, 16)), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        L.orthogonalize(x, x, torch.zeros(8, dtype=torch.uint8))


def test_kernel_kinds_have_names(L):
    names = [L.moe_profile_kernel_name(i) for i in range(64)]
    known = [n for n in names if n]
    assert len(set(known)) == len(known) and names[len(known):] == [None] * (64 - len(known))
    assert {"join_fwd", "join_bwd", "route_bwd", "orth_load", "orth_steps", "orth_small"} <= set(known)
