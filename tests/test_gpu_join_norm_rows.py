"""Joining norms where a block walks many rows and where a row's columns choose another
form: the middle widths of the backward, and gates and 1 / rms values, which a warp keeps
for 32 rows at a time, over several such windows.  Bounds: test_gpu_join_norm.py."""

import pytest
import torch

from test_gpu_join_norm import DT, Case, Grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 4104), (5, 8192), (2, 6000), (700, 5152), (400, 8184), (330, 4608)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_of_middle_widths(T, H, dtype):
    """4104 to 8192 columns: two vectors a thread in bf16, the row read twice where it goes
    through shared memory; clusters in fp32."""
    Grad(T, H, DT[dtype]).check_bwd()
    Grad(T, H, DT[dtype], next_norm=False, scale=0.5).check_bwd()
    Grad(T, H, DT[dtype], d_total=False, post_weight=False, gate=False).check_bwd()
    c = Grad(T, H, DT[dtype], post_norm=False, scale=1.5)
    a, b = c.check_bwd(), c.run_bwd()
    assert all(torch.equal(a[k], b[k]) for k in a)
    for where in (dict(dy="dn", d_residual="y"), dict(dy="total", d_residual="d_total")):
        got = c.run_bwd(**where)
        assert all(torch.equal(a[k], got[k]) for k in a)


class OnGpu:
    """The reference in 64 bits on the GPU: many rows take long on the host."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.move()

    def move(self):
        for k, v in vars(self).items():
            if isinstance(v, torch.Tensor):
                setattr(self, k, v.cuda())

    def exact(self):
        self.move()
        return super().exact()

    def run(self, *a, **kw):
        return {k: v.cuda() for k, v in super().run(*a, **kw).items()}


class GpuCase(OnGpu, Case):
    pass


class GpuGrad(OnGpu, Grad):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.move()

    def grads(self):
        # (the parent makes zeros on the host where there is no d_total)
        assert self.d_total is not None
        return super().grads()

    def run_bwd(self, *a, **kw):
        return {k: v.cuda() for k, v in super().run_bwd(*a, **kw).items()}


@pytest.mark.parametrize("T,H", [(20001, 2880), (11001, 4104)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", ["same", "e4m3", ""])
def test_forward_of_many_rows_per_block(T, H, dtype, norm):
    if norm == "e4m3":
        H -= H % 32
    GpuCase(T, H, DT[dtype]).check(norm)


@pytest.mark.parametrize("T,H", [(10001, 3000), (12000, 4096), (5200, 6000), (2600, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_of_many_rows_per_block(T, H, dtype):
    GpuGrad(T, H, DT[dtype]).check_bwd()
    GpuGrad(T, H, DT[dtype], next_norm=False, scale=0.5).check_bwd()
