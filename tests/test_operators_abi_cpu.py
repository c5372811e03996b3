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


def test_grad_clip_refusals(L):
    def table(*entries):
        return (L.MoeGrad * len(entries))(*[L.MoeGrad(*e) for e in entries])

    good = table((16, 16, 5, L.MOE_FP32), (18, 34, 7, L.MOE_BF16), (None, None, 0, L.MOE_FP32))
    size = L.moe_grad_clip_workspace_size(good, 3)
    assert size > 0 and L.moe_grad_clip_workspace_size(None, 0) > 0
    for bad in (table((None, 16, 5, L.MOE_FP32)), table((18, 16, 5, L.MOE_FP32)),
                table((16, 18, 5, L.MOE_FP32)), table((17, 16, 5, L.MOE_BF16)),
                table((16, 16, -1, L.MOE_FP32)), table((16, 16, 5, 9))):
        assert L.moe_grad_clip_workspace_size(bad, 1) == 0
        assert L.moe_grad_clip(bad, 1, 1.0, 16, 256, 1 << 30, None) == L.MOE_ERR_INVALID_ARG
    args = dict(grads=good, n=3, max_norm=1.0, norm_out=16, ws=256, ws_bytes=size, stream=None)
    for bad in (dict(n=-1), dict(grads=None), dict(max_norm=-1.0), dict(max_norm=float("nan")),
                dict(norm_out=None), dict(norm_out=18), dict(ws=None), dict(ws=272)):
        assert L.moe_grad_clip(**dict(args, **bad)) == L.MOE_ERR_INVALID_ARG, bad
    assert L.moe_grad_clip(**dict(args, ws_bytes=size - 1)) == L.MOE_ERR_WORKSPACE
    many = table(*[(16, 16, 5, L.MOE_FP32)] * 200)
    assert L.moe_grad_clip_workspace_size(many, 200) > size


def test_mx_refusals(L):
    ok = dict(w=16, dtype=L.MOE_BF16, E=2, K=64, N=16, codes=16, scales=1, stream=None)
    for bad in (dict(K=48), dict(K=0), dict(N=12), dict(N=0), dict(E=-1), dict(dtype=5),
                dict(w=None), dict(codes=None), dict(scales=None), dict(w=8), dict(codes=8),
                dict(E=1 << 40)):
        assert L.moe_mx_quantize(**dict(ok, **bad)) == L.MOE_ERR_INVALID_ARG, bad
        assert L.moe_mx_dequantize(**dict(ok, **bad)) == L.MOE_ERR_INVALID_ARG, bad
    assert L.moe_mx_quantize(**dict(ok, E=0, w=None, codes=None, scales=None)) == L.MOE_OK
    assert L.moe_mx_quantize(**dict(ok, E=0, K=48)) == L.MOE_ERR_INVALID_ARG


def test_grad_struct_layout(L, tmp_path):
    import ctypes
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "g.c", tmp_path / "g"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {'
                   'printf("%zu %zu %zu %zu %zu", sizeof(moe_grad_t), offsetof(moe_grad_t, src),'
                   'offsetof(moe_grad_t, dst), offsetof(moe_grad_t, n), offsetof(moe_grad_t, dtype));'
                   'return 0; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(L.MoeGrad)] + [getattr(L.MoeGrad, f).offset
                                                for f in ("src", "dst", "n", "dtype")]


def test_ffn_few_refusals(L):
    s = L.Shape(4, 64, 64, 8, 2)
    size = L.moe_few_workspace_size(s)
    assert size >= 8 * 64 * 2 + 8 * 64 * 4
    assert L.moe_few_workspace_size(L.Shape(128, 64, 64, 8, 2)) > size
    for bad in (dict(T=129), dict(H=12), dict(T=-1)):
        assert L.moe_few_workspace_size(L.Shape(**dict(dict(T=4, H=64, I=64, E=8, k=2), **bad))) == 0
    ok = dict(shape=s, x=16, x_scale=None, topk_idx=16, topk_w=16, w_gate_up=16, w_down=16, mx=None,
              bias=None, y=16, ws=256, ws_bytes=size, stream=None)
    mx = L.MoeMxWeights(16, 1, 16, 1)
    for bad in (dict(x=None), dict(topk_idx=None), dict(topk_w=None), dict(w_gate_up=None),
                dict(w_down=None), dict(y=None), dict(ws=None), dict(ws=128), dict(x=8), dict(y=8),
                dict(w_gate_up=8), dict(w_down=8), dict(mx=mx),
                dict(bias=L.MoeBias(8, None, None, None)),
                dict(w_gate_up=None, w_down=None, mx=L.MoeMxWeights(16, None, 16, 1)),
                dict(w_gate_up=None, w_down=None, mx=L.MoeMxWeights(16, 1, 8, 1)),
                dict(w_gate_up=None, w_down=None, mx=mx, shape=L.Shape(4, 64, 40, 8, 2)),
                dict(w_gate_up=None, w_down=None, mx=mx, shape=L.Shape(4, 72, 64, 8, 2)),
                dict(x_scale=1, shape=L.Shape(4, 72, 64, 8, 2))):
        assert L.moe_ffn_few(**dict(ok, **bad)) == L.MOE_ERR_INVALID_ARG, bad
    assert L.moe_ffn_few(**dict(ok, ws_bytes=size - 1)) == L.MOE_ERR_WORKSPACE
    assert L.moe_ffn_few(**dict(ok, shape=L.Shape(129, 64, 64, 8, 2))) == L.MOE_ERR_UNSUPPORTED
    f32 = L.Shape(4, 64, 64, 8, 2, dtype=L.MOE_FP32)
    assert L.moe_ffn_few(**dict(ok, shape=f32, w_gate_up=None, w_down=None, mx=mx)) == L.MOE_ERR_UNSUPPORTED
    assert L.moe_ffn_few(**dict(ok, shape=L.Shape(0, 64, 64, 8, 2), x=None, y=None)) == L.MOE_OK
