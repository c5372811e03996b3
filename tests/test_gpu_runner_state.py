"""What LayerRunner keeps between calls: bias gradients of an earlier backward,
buffers made at a call on another stream, 4-bit weights and clipping workspaces
that a captured graph still uses."""

import pytest
import torch

import dispatch_gemm_combine_gb300 as moe
from dispatch_gemm_combine_gb300.runner import LayerRunner

pytestmark = pytest.mark.gpu

H, I, E, K = 96, 64, 4, 2


def inputs(T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def bf16(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)

    idx = torch.topk(torch.randn((T, E), generator=g, device="cuda"), K, dim=-1).indices.to(torch.int32)
    w = torch.full((T, K), 0.5, device="cuda")
    return dict(x=bf16(T, H), idx=idx.contiguous(), w=w, wgu=bf16(E, H, 2 * I, std=0.1),
                wd=bf16(E, I, H, std=0.1), dy=bf16(T, H), bgu=bf16(E, 2 * I, std=0.1), bd=bf16(E, H, std=0.1))


def train(r, d, bias):
    a = [d[n] for n in ("x", "idx", "w", "wgu", "wd")]
    b = dict(b_gate_up=d["bgu"], b_down=d["bd"]) if bias else {}
    r.plan(d["idx"])
    r.forward(*a, **b)
    r.backward(d["dy"], *a, **b)


def test_clip_grads_takes_the_last_backwards_gradients():
    d = inputs(40)
    r = LayerRunner(40, H, I, E, K, moe.MOE_ACT_SWIGLU)
    train(r, d, True)
    norm = r.clip_grads(float("inf"))[0].item()
    ref = sum(float(t.double().square().sum()) for t in (r.dw_gate_up, r.dw_down, r.db_gate_up, r.db_down)) ** 0.5
    assert abs(norm - ref) <= 1e-6 * ref
    stale = r.db_gate_up.clone(), r.db_down.clone()
    train(r, d, False)
    ref = sum(float(t.double().square().sum()) for t in (r.dw_gate_up, r.dw_down)) ** 0.5
    norm = r.clip_grads(0.25 * ref)
    assert abs(norm[0].item() - ref) <= 1e-6 * ref
    assert torch.equal(r.db_gate_up, stale[0]) and torch.equal(r.db_down, stale[1])
    train(r, d, True)
    ref = sum(float(t.double().square().sum()) for t in (r.dw_gate_up, r.dw_down, r.db_gate_up, r.db_down)) ** 0.5
    assert abs(r.clip_grads(float("inf"))[0].item() - ref) <= 1e-6 * ref


def test_first_few_on_another_stream_keeps_its_error():
    d = inputs(3)
    r = LayerRunner(3, H, I, E, K, moe.MOE_ACT_SWIGLU, training=False, backward=False)
    d["idx"][1, 1] = E
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)         # what the current stream still has to do
    r.few(*[d[n] for n in ("x", "idx", "w", "wgu", "wd")], stream=s)
    torch.cuda.synchronize()
    with pytest.raises(moe.MoeError) as e:
        r.check()
    assert e.value.status == moe.MOE_ERR_BAD_INDEX


def test_buffers_made_at_a_call_are_its_streams():
    """... so that what the allocator hands out has no work of another stream pending."""
    d = inputs(40)
    r = LayerRunner(40, H, I, E, K, moe.MOE_ACT_SWIGLU)
    s = torch.cuda.Stream()
    many = [torch.ones(3, device="cuda") for _ in range(300)]
    torch.cuda.synchronize()
    a = [d[n] for n in ("x", "idx", "w", "wgu", "wd")]
    bias = dict(b_gate_up=d["bgu"], b_down=d["bd"])
    r.plan(d["idx"], stream=s)
    r.forward(*a, stream=s, **bias)
    r.backward(d["dy"], *a, recompute=True, stream=s, **bias)
    r.clip_grads(1.0, extra=many, stream=s)
    r.quantize(d["wgu"], d["wd"], stream=s)
    torch.cuda.synchronize()
    made = [r.ws_bwd_recompute, r.db_gate_up, r.db_down, r.ws_clip, *r.mx_t]
    for t in made:
        at = [g for g in torch.cuda.memory_snapshot()
              if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert len(at) == 1 and at[0]["stream"] == s.cuda_stream


def test_quantizing_again_serves_the_new_weights_in_a_captured_graph():
    d, new = inputs(5), inputs(5, seed=1)
    r = LayerRunner(5, H, I, E, K, moe.MOE_ACT_SWIGLU, training=False, backward=False)
    first = r.quantize(d["wgu"], d["wd"])
    at = [t.data_ptr() for t in first]
    a = [d[n] for n in ("x", "idx", "w")]
    r.few(*a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.few(*a)
    second = r.quantize(new["wgu"], new["wd"])
    assert [t.data_ptr() for t in second] == at
    fresh = LayerRunner(5, H, I, E, K, moe.MOE_ACT_SWIGLU, training=False, backward=False)
    fresh.quantize(new["wgu"], new["wd"])
    right = fresh.few(*a)
    r.y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.y, right)


def test_clip_grads_with_lists_that_grow():
    d = inputs(40)
    r = LayerRunner(40, H, I, E, K, moe.MOE_ACT_SWIGLU)
    train(r, d, False)
    kept = r.dw_gate_up.clone(), r.dw_down.clone()
    norm = r.clip_grads(1e-3)
    right = norm.clone()
    scaled = r.dw_gate_up.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.clip_grads(1e-3)
    for n in (90, 250, 400):      # one launch's tensors, several, more
        extra = [torch.full((5,), 2.0, device="cuda") for _ in range(n)]
        r.dw_gate_up.copy_(kept[0]), r.dw_down.copy_(kept[1])
        out = r.clip_grads(float("inf"), extra=extra)
        ref = (float(kept[0].double().square().sum()) + float(kept[1].double().square().sum()) + 20.0 * n) ** 0.5
        assert abs(out[0].item() - ref) <= 1e-6 * ref
        assert out.data_ptr() == norm.data_ptr()
    # a list with empty entries, then a shorter one without
    r.clip_grads(1.0, extra=[torch.empty(0, device="cuda")] * 900)
    r.clip_grads(1.0, extra=[torch.ones(1, device="cuda")] * 500)
    r.dw_gate_up.copy_(kept[0]), r.dw_down.copy_(kept[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, right) and torch.equal(r.dw_gate_up, scaled)
