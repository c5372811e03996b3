"""What the torch helpers of the operators refuse before the library is called: here
with stand-ins for GPU tensors and a library that only records its calls."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe

T, H, I, E, K = 3, 128, 64, 4, 2


class Fake:
    """What the helpers ask of a tensor."""

    def __init__(self, shape, dtype, is_cuda=True):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, is_cuda

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return moe.MOE_OK
        return call


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    return r


def u8(*shape):
    return Fake(shape, torch.uint8)


def bf16(*shape):
    return Fake(shape, torch.bfloat16)


def few(library, mx=None, bias=None, ws=None):
    dense = () if mx else (bf16(E, H, 2 * I), bf16(E, I, H))
    moe.ffn_few(moe.Shape(T, H, I, E, K), bf16(T, H), Fake((T, K), torch.int32), Fake((T, K), torch.float32),
                *(dense or (None, None)), bf16(T, H), u8(1 << 20) if ws is None else ws, bias=bias, mx=mx)
    return library.calls


GOOD = dict(codes_gate_up=(E, 2 * I, H // 2), scales_gate_up=(E, 2 * I, H // 32),
            codes_down=(E, H, I // 2), scales_down=(E, H, I // 32))


def test_4bit_weights_of_the_layers_shape_are_taken(library):
    assert few(library, moe.mx_struct(*[u8(*s) for s in GOOD.values()])) == ["moe_ffn_few"]


@pytest.mark.parametrize("name,shape", [
    ("codes_gate_up", (E - 1, 2 * I, H // 2)), ("codes_gate_up", (E, 2 * I, H // 4)),
    ("codes_gate_up", (E, I, H // 2)), ("codes_gate_up", (E * 2 * I, H // 2)),
    ("scales_gate_up", (E, 2 * I, H // 64)), ("scales_gate_up", (E, I, H // 32)),
    ("scales_gate_up", (E - 1, 2 * I, H // 32)), ("codes_down", (E, H, I // 4)),
    ("codes_down", (E, H // 2, I // 2)), ("scales_down", (E, H, 1)), ("scales_down", (E - 1, H, I // 32))])
def test_4bit_weights_of_another_shape_are_refused(library, name, shape):
    with pytest.raises(ValueError):
        few(library, moe.mx_struct(*[u8(*s) for s in dict(GOOD, **{name: shape}).values()]))
    assert library.calls == []


def test_exchanged_projections_are_refused(library):
    a, b, c, d = [u8(*s) for s in GOOD.values()]
    for ts in ((c, d, a, b), (a, d, c, b), (b, a, d, c)):
        with pytest.raises(ValueError):
            few(library, moe.mx_struct(*ts))
    assert library.calls == []


def test_structs_keep_their_tensors(library):
    import gc
    import weakref
    ts = [u8(*s) for s in GOOD.values()]
    refs = [weakref.ref(t) for t in ts]
    s = moe.mx_struct(*ts)
    del ts
    gc.collect()
    assert all(r() is not None for r in refs) and s is not None
    b = [bf16(E, 2 * I), bf16(E, H)]
    refs = [weakref.ref(t) for t in b]
    s = moe.bias_struct(*b)
    del b
    gc.collect()
    assert all(r() is not None for r in refs) and s is not None


@pytest.mark.parametrize("b_gate_up,b_down", [
    (bf16(E, I), None), (bf16(E - 1, 2 * I), None), (Fake((E, 2 * I), torch.float32), None),
    (None, bf16(E, I)), (None, Fake((E, H), torch.bfloat16, False))])
def test_biases_of_another_kind_are_refused(library, b_gate_up, b_down):
    assert few(library, bias=moe.bias_struct(bf16(E, 2 * I), bf16(E, H))) == ["moe_ffn_few"]
    library.calls.clear()
    with pytest.raises(ValueError):
        few(library, bias=moe.bias_struct(b_gate_up, b_down))
    assert library.calls == []


def test_workspaces_on_the_host_are_refused(library):
    host = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        few(library, ws=host)
    table = (moe.MoeGrad * 1)()
    table.count = 0
    with pytest.raises(ValueError):
        moe.grad_clip(table, 1.0, Fake((2,), torch.float32), host)
    with pytest.raises(ValueError):
        moe.rms_norm_bwd(bf16(T, H), bf16(T, H), Fake((T,), torch.float32), bf16(H), bf16(T, H),
                         Fake((H,), torch.float32), ws=host)
    assert library.calls == []
    moe.rms_norm_bwd(bf16(T, H), bf16(T, H), Fake((T,), torch.float32), bf16(H), bf16(T, H))
    assert library.calls == ["moe_rms_norm_bwd"]
