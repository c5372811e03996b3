"""Host-side checks of the operators around the layer: what their C entry
points refuse before any device access, and their workspace sizes."""

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from dispatch_gemm_combine_gb300 import _build
    _build.build()
    import dispatch_gemm_combine_gb300 as m
    return m


def test_rms_norm_refusals(L):
    ok = dict(T=4, H=64, dtype=L.MOE_BF16, x=16, residual=None, weight=16, eps=1e-6, y=16,
              y_scale=None, total=None, rstd=None, stream=None)
    bad = [dict(H=12), dict(H=0), dict(H=40000), dict(T=-1), dict(T=1 << 31), dict(dtype=7),
           dict(x=None), dict(weight=None), dict(y=None), dict(x=24), dict(residual=8),
           dict(weight=20), dict(y=8), dict(total=8), dict(eps=-1.0), dict(eps=float("nan")),
           dict(H=40, y_scale=16)]
    for b in bad:
        assert L.moe_rms_norm_fwd(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    assert L.moe_rms_norm_fwd(**dict(ok, T=0, x=None, y=None)) == L.MOE_OK
    ok = dict(T=4, H=64, dtype=L.MOE_BF16, dy=16, d_total=None, total=16, rstd=16, weight=16, dx=16,
              dweight=16, ws=256, ws_bytes=1 << 30, stream=None)
    bad = [dict(H=12), dict(T=-1), dict(dtype=2), dict(dy=None), dict(total=None), dict(rstd=None),
           dict(weight=None), dict(dx=None), dict(dy=8), dict(d_total=8), dict(total=8),
           dict(dx=8), dict(dweight=8), dict(ws=None), dict(ws=16)]
    for b in bad:
        assert L.moe_rms_norm_bwd(**dict(ok, **b)) == L.MOE_ERR_INVALID_ARG, b
    need = L.moe_rms_norm_workspace_size(4, 64)
    assert need >= 4 * 64 * 4
    assert L.moe_rms_norm_bwd(**dict(ok, ws_bytes=need - 1)) == L.MOE_ERR_WORKSPACE
    assert L.moe_rms_norm_workspace_size(4, 65) == 0 and L.moe_rms_norm_workspace_size(-1, 64) == 0


def test_rms_norm_helper_refusals(L):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):           # not on the GPU
        L.rms_norm_fwd(x, w, x)
    with pytest.raises(ValueError):           # a type that is not held
        L.rms_norm_fwd(x.double(), w, x)
