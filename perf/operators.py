"""Cases for the operators around the expert layer, and their plain forms.

Four operators are measured, as a transformer block with an expert layer uses
them:

  norm_fwd, norm_bwd   RMS norm with the residual's addition; the output in the
                       storage type or as e4m3 with one power-of-two scale per
                       32 columns; the backward with the weight's gradient
  few                  the whole expert layer for a few tokens: bf16, fp32 or
                       4-bit (microscaled) expert weights, tokens in the
                       storage type or as e4m3 with scales
  mx                   microscaled 4-bit weights: quantisation of [E, K, N]
                       expert weights along K and back (the round trip), or
                       the way back alone
  clip                 the global norm of many gradients, and clipping by it

`run` computes a case in elementary torch operations (own = False) or calls
dispatch_gemm_combine_gb300 (own = True).  `exact` computes it in 64 bits.

Microscaled blocks: 32 consecutive values share the scale 2^q, the smallest
power of two (q in [-127, 127]) with amax <= 448 * 2^q for e4m3 and
amax <= 6 * 2^q for e2m1; the codes are the values divided by it, rounded to
nearest, ties to even.  The scale byte is q + 127.
"""

import math

import torch

own = False

CLAMPED, SWIGLU = 1, 0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _few(name, T, H, I, E, k, act, weights, bias=False, x8=False, interleaved=False):
    return {"name": name, "op": "few", "T": T, "H": H, "I": I, "E": E, "k": k, "act": act,
            "weights": weights, "bias": bias, "x8": x8, "interleaved": interleaved}


def _norm(name, T, H, dtype, residual=True, out8=False, train=False):
    return {"name": name, "op": "norm_fwd", "T": T, "H": H, "dtype": dtype, "residual": residual,
            "out8": out8, "train": train}


def _norm_bwd(name, T, H, dtype, d_total=True):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "dtype": dtype, "d_total": d_total}


def _mx(name, E, K, N, dtype, back_only=False):
    return {"name": name, "op": "mx", "E": E, "K": K, "N": N, "dtype": dtype,
            "back_only": back_only}


def _clip(name, count, largest, E, H, I, dtype, clipped=True):
    """`count` gradients of ragged sizes up to `largest`, and with E > 0 the two
    weight gradients of an expert layer."""
    return {"name": name, "op": "clip", "count": count, "largest": largest, "E": E, "H": H, "I": I,
            "dtype": dtype, "clipped": clipped}


def listed():
    return [
        # one token decoded by the layer with H = I = 2880, 128 experts, top-4
        _few("few_one_bf16", 1, 2880, 2880, 128, 4, CLAMPED, "bf16", bias=True),
        # a small serving batch on the layer with H = 4096, I = 2048, 256 experts, top-8
        _few("few_batch16_bf16", 16, 4096, 2048, 256, 8, SWIGLU, "bf16"),
        # the tiny single-precision layer: all latency
        _few("few_tiny_fp32", 5, 128, 128, 8, 2, SWIGLU, "fp32", interleaved=True),
        # one token with 4-bit expert weights and the norm's 8-bit output as input
        _few("few_one_mx", 1, 2880, 2880, 128, 4, CLAMPED, "mx", bias=True, x8=True),
        # a serving batch on one rank's share (64 experts) of the H = 8192 layer, 4-bit weights:
        # a few rows for each expert
        _few("few_batch32_mx", 32, 8192, 2048, 64, 8, SWIGLU, "mx"),
        # the gate_up weights of 16 experts of the H = I = 2880 layer, quantised and read back
        _mx("mx_round_trip_gate_up", 16, 2880, 5760, "bf16"),
        # ragged small weights in single precision, from codes back to values
        _mx("mx_back_small", 3, 416, 200, "fp32", back_only=True),
        # one decoded token: norm of the residual stream
        _norm("norm_one", 1, 2880, "bf16"),
        # a long prompt, handed to the expert layer in 8 bits
        _norm("norm_long_e4m3", 16384, 4096, "bf16", out8=True),
        # the training backward at the benchmark's size
        _norm_bwd("norm_bwd_train", 8192, 2880, "bf16"),
        # the small parameters of a block: ragged sizes, latency
        _clip("clip_small", 12, 5000, 0, 0, 0, "fp32"),
        # one rank's expert gradients (32 experts of the H = I = 2880 layer) and small ones
        _clip("clip_layer", 6, 40000, 32, 2880, 2880, "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "few", "mx", "norm_fwd", "norm_fwd", "norm_bwd", "clip"])
    if op == "few":
        weights = rng.choice(["bf16", "bf16", "mx", "mx", "fp32"])
        step = 32 if weights == "mx" else 8
        x8 = weights == "mx" and rng.random() < 0.5
        top = 1024 if weights == "fp32" else 4096
        H, I = (step * max(1, _log(rng, 64, top) // step) for _ in range(2))
        k = rng.choice([1, 2, 4, 6, 8])
        # no more slots' products, and no more weights, than the largest listed case
        E = max(k, min(_log(rng, 4, 64), 800_000_000 // (H * I)))
        T = min(_log(rng, 1, 64), max(1, 1_000_000_000 // (k * H * I)))
        c = _few("", T, H, I, E, k, rng.choice([CLAMPED, SWIGLU]), weights,
                 rng.random() < 0.4, x8, rng.random() < 0.3)
    elif op == "mx":
        back = rng.random() < 0.5
        c = _mx("", _log(rng, 1, 16), 32 * _log(rng, 1, 90), 8 * _log(rng, 1, 500),
                rng.choice(["bf16", "bf16", "fp32"]), back)
    elif op == "norm_fwd":
        out8 = rng.random() < 0.4
        step = 32 if out8 else 8
        c = _norm("", _log(rng, 1, 16384), step * max(1, _log(rng, 64, 8192) // step),
                  rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7, out8,
                  rng.random() < 0.5)
    elif op == "norm_bwd":
        c = _norm_bwd("", _log(rng, 1, 8192), 8 * max(1, _log(rng, 64, 8192) // 8),
                      rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.6)
    else:
        layer = rng.random() < 0.5
        c = _clip("", _log(rng, 1, 40), _log(rng, 10, 1000000), _log(rng, 1, 16) if layer else 0,
                  8 * _log(rng, 8, 256) if layer else 0, 8 * _log(rng, 8, 256) if layer else 0,
                  rng.choice(["fp32", "fp32", "bf16"]), rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _randn(g, shape, dtype=torch.float32, std=1.0):
    v = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return v if std == 1.0 else v.mul_(std)


_PAIRS = {}


def _code_pairs(g, shape):
    """Packed e2m1 codes as quantised normal weights have them: a byte holds two
    independent codes, drawn from a table of 65536 pairs."""
    if not _PAIRS:
        t = torch.Generator(device="cuda").manual_seed(11)
        v = torch.randn((2, 65536), generator=t, device="cuda") * 2.2
        code = _e2m1_code(v)
        _PAIRS["table"] = (code[0] | (code[1] << 4)).to(torch.uint8)
    at = torch.randint(0, 65536, shape, generator=g, device="cuda", dtype=torch.int32)
    return _PAIRS["table"][at]


def _scale_bytes(g, shape):
    return torch.randint(118, 122, shape, generator=g, device="cuda", dtype=torch.uint8)


def _prepare_few(c, g):
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    dt = torch.float32 if c["weights"] == "fp32" else torch.bfloat16
    s = {"case": c}
    x = _randn(g, (T, H))
    if c["x8"]:
        code, byte = _to_e4m3(x)
        s["x"], s["x_scale"] = code.view(torch.uint8), byte
    else:
        s["x"] = x.to(dt)
    top = torch.topk(_randn(g, (T, E)), k, dim=-1)
    s["idx"] = top.indices.to(torch.int32).contiguous()
    s["w"] = torch.softmax(top.values, dim=-1)
    if c["weights"] == "mx":
        s["mx"] = (_code_pairs(g, (E, 2 * I, H // 2)), _scale_bytes(g, (E, 2 * I, H // 32)),
                   _code_pairs(g, (E, H, I // 2)), _scale_bytes(g, (E, H, I // 32)))
    else:
        s["w_gate_up"] = _randn(g, (E, H, 2 * I), dt, 0.02)
        s["w_down"] = _randn(g, (E, I, H), dt, 0.02)
    if c["bias"]:
        s["b_gate_up"] = _randn(g, (E, 2 * I), dt, 0.5)
        s["b_down"] = _randn(g, (E, H), dt, 0.5)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "few":
        return _prepare_few(case, g)
    s = {"case": case}
    if op == "mx":
        E, K, N = case["E"], case["K"], case["N"]
        if case["back_only"]:
            s["codes"], s["scales"] = _code_pairs(g, (E, N, K // 2)), _scale_bytes(g, (E, N, K // 32))
        else:
            s["w"] = _randn(g, (E, K, N), _dtype(case), 0.02)
    elif op in ("norm_fwd", "norm_bwd"):
        T, H, dt = case["T"], case["H"], _dtype(case)
        s["weight"] = (1 + _randn(g, (H,), std=0.1)).to(dt)
        x = _randn(g, (T, H))
        if op == "norm_fwd":
            s["x"] = x.to(dt)
            if case["residual"]:
                s["residual"] = _randn(g, (T, H), std=3.0).to(dt)
        else:
            s["total"] = (3 * x).to(dt)
            s["rstd"] = torch.rsqrt(s["total"].float().square().mean(-1) + 1e-6)
            s["dy"] = _randn(g, (T, H)).to(dt)
            if case["d_total"]:
                s["d_total"] = _randn(g, (T, H)).to(dt)
    else:
        dt = _dtype(case)
        # the sizes are the case's, whatever the seed
        sizes = torch.randint(1, case["largest"] + 1, (case["count"],),
                              generator=torch.Generator().manual_seed(3)).tolist()
        s["grads"] = [_randn(g, (n,), dt, 0.01) for n in sizes]
        if case["E"]:
            E, H, I = case["E"], case["H"], case["I"]
            s["grads"] += [_randn(g, (E, H, 2 * I), dt, 0.01), _randn(g, (E, I, H), dt, 0.01)]
        n = sum(t.numel() for t in s["grads"])
        # the norm is near 0.01 sqrt(n): a limit on either side of it
        s["max_norm"] = 0.01 * math.sqrt(n) * (0.3 if case["clipped"] else 3.0)
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ------------------------------------------------------------------ plain forms
def _pow2(q):
    """2^q in 32 bits from whole q in [-126, 127] (bits of the exponent field)."""
    return ((q + 127) << 23).view(torch.float32)


def _block_exponent(v, top_fraction, top_exponent):
    """q of each block of 32 (last axis): the smallest with amax <= top * 2^q,
    top = top_fraction * 2^top_exponent."""
    amax = v.abs().amax(-1)
    frac, exp = torch.frexp(amax)
    q = exp.to(torch.int32) - top_exponent + (frac > top_fraction).to(torch.int32)
    return torch.where(amax == 0, torch.full_like(q, -127), q.clamp(-127, 127))


def _scaled(v, q):
    """v * 2^-q without leaving the range of the type on the way."""
    half = torch.div(q, 2, rounding_mode="floor")
    return v * _pow2(-half)[..., None].to(v.dtype) * _pow2(half - q)[..., None].to(v.dtype)


def _to_e4m3(v):
    """(codes as float8_e4m3fn, scale bytes) of v [..., H]."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    q = _block_exponent(b, 0.875, 9)
    code = _scaled(b, q).to(torch.float32).to(torch.float8_e4m3fn)
    return code.reshape(v.shape), (q + 127).to(torch.uint8)


def _e2m1_code(v):
    """e2m1 codes 0..15 (sign in bit 3) of v, ties to even."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _mx_values(codes, scales):
    """[..., K/2] codes and [..., K/32] scale bytes -> values [..., K] in 32 bits."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1)
    v = v.reshape(*scales.shape, 32) * _pow2(scales.to(torch.int32) - 127)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _x8_values(code, byte):
    v = code.view(torch.float8_e4m3fn).float().reshape(*byte.shape, 32)
    return (v * _pow2(byte.to(torch.int32) - 127)[..., None]).reshape(code.shape)


def _plain_few(s):
    c = s["case"]
    I = c["I"]
    x = _x8_values(s["x"], s["x_scale"]) if c["x8"] else s["x"].float()
    y = torch.zeros((c["T"], c["H"]), device=x.device)
    for j in range(c["k"]):                      # y = sum over the k choices, j ascending
        e = s["idx"][:, j].long()
        if c["weights"] == "mx":
            cg, sg, cd, sd = s["mx"]
            h = torch.bmm(_mx_values(cg[e], sg[e]), x[:, :, None])[:, :, 0]
        else:
            h = torch.bmm(x[:, None, :], s["w_gate_up"][e].float())[:, 0]
        if c["bias"]:
            h = h + s["b_gate_up"][e].float()
        gate, up = (h[:, 0::2], h[:, 1::2]) if c["interleaved"] else (h[:, :I], h[:, I:])
        if c["act"] == CLAMPED:
            gate, up = gate.clamp(max=7.0), up.clamp(-7.0, 7.0)
            a = (up + 1) * gate * torch.sigmoid(1.702 * gate)
        else:
            a = gate * torch.sigmoid(gate) * up
        if c["weights"] == "mx":
            o = torch.bmm(_mx_values(cd[e], sd[e]), a[:, :, None])[:, :, 0]
        else:
            o = torch.bmm(a[:, None, :], s["w_down"][e].float())[:, 0]
        if c["bias"]:
            o = o + s["b_down"][e].float()
        y += s["w"][:, j:j + 1] * o
    return {"y": y.to(torch.float32 if c["weights"] == "fp32" else torch.bfloat16)}


def _plain_norm(s):
    c = s["case"]
    dt = _dtype(c)
    # the 8-bit output rounds and scales by borders: 64 bits up to there
    wide = torch.float64 if c["out8"] else torch.float32
    r = s["x"].to(wide)
    if c["residual"]:
        r = r + s["residual"].to(wide)
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6)
    y = r * rstd * s["weight"].to(wide)
    out = {}
    if c["out8"]:
        out["y"], byte = _to_e4m3(y)
        out["y_scale"] = byte.view(torch.float8_e8m0fnu)
    else:
        out["y"] = y.to(dt)
    if c["residual"]:
        out["total"] = r.to(dt)
    if c["train"]:
        out["rstd"] = rstd[:, 0].float()
    return out


def _plain_norm_bwd(s):
    r, rstd = s["total"].float(), s["rstd"][:, None]
    dy = s["dy"].float()
    xhat = r * rstd
    dn = dy * s["weight"].float()
    dx = rstd * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
    if s["case"]["d_total"]:
        dx = dx + s["d_total"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).double().sum(0).float()}


def _plain_mx(s):
    c = s["case"]
    if c["back_only"]:
        return {"w": _mx_values(s["codes"], s["scales"]).transpose(1, 2).to(_dtype(c)).contiguous()}
    b = s["w"].transpose(1, 2).float().reshape(c["E"], c["N"], c["K"] // 32, 32)
    q = _block_exponent(b, 0.75, 3)
    code = _e2m1_code(_scaled(b, q)).reshape(c["E"], c["N"], c["K"] // 2, 2)
    byte = (q + 127).to(torch.uint8)
    w = _mx_values(code[..., 0] | (code[..., 1] << 4), byte)
    return {"w": w.transpose(1, 2).to(_dtype(c)).contiguous(),
            "scales": byte.view(torch.float8_e8m0fnu)}


def _plain_clip(s):
    total = sum(t.double().square().sum() for t in s["grads"])
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
    return {"norm": norm.float(), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


# ------------------------------------------------------------------ the framework's operators
def _own_few(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    if "shape" not in s:      # what a program keeps between calls: the shape, the workspace, y
        fp32 = c["weights"] == "fp32"
        s["shape"] = moe.Shape(c["T"], c["H"], c["I"], c["E"], c["k"], c["act"],
                               moe.MOE_FP32 if fp32 else moe.MOE_BF16, 7.0, 1.702,
                               1 if c["interleaved"] else 0)
        s["ws"] = moe.few_workspace(s["shape"])
        s["y"] = torch.empty((c["T"], c["H"]), device="cuda",
                             dtype=torch.float32 if fp32 else torch.bfloat16)
        s["bias"] = moe.bias_struct(s.get("b_gate_up"), s.get("b_down"))
        s["mx_struct"] = moe.mx_struct(*s["mx"]) if "mx" in s else None
    moe.ffn_few(s["shape"], s["x"], s["idx"], s["w"], s.get("w_gate_up"), s.get("w_down"), s["y"],
                s["ws"], bias=s["bias"], x_scale=s.get("x_scale"), mx=s["mx_struct"])
    return {"y": s["y"]}


def _own_norm(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    if "y" not in s:
        T, H = c["T"], c["H"]
        s["y"] = torch.empty((T, H), device="cuda", dtype=torch.uint8 if c["out8"] else _dtype(c))
        s["y_scale"] = (torch.empty((T, H // 32), device="cuda", dtype=torch.uint8)
                        if c["out8"] else None)
        s["sum"] = torch.empty((T, H), device="cuda", dtype=_dtype(c)) if c["residual"] else None
        s["rs"] = torch.empty(T, device="cuda", dtype=torch.float32) if c["train"] else None
    moe.rms_norm_fwd(s["x"], s["weight"], s["y"], eps=1e-6, residual=s.get("residual"),
                     total=s["sum"], rstd=s["rs"], y_scale=s["y_scale"])
    out = {"y": s["y"].view(torch.float8_e4m3fn) if c["out8"] else s["y"]}
    if c["out8"]:
        out["y_scale"] = s["y_scale"].view(torch.float8_e8m0fnu)
    if c["residual"]:
        out["total"] = s["sum"]
    if c["train"]:
        out["rstd"] = s["rs"]
    return out


def _own_norm_bwd(s):
    import dispatch_gemm_combine_gb300 as moe
    if "dx" not in s:
        s["dx"] = torch.empty_like(s["dy"])
        s["dweight"] = torch.empty(s["case"]["H"], device="cuda", dtype=torch.float32)
        s["ws"] = moe.rms_norm_workspace(s["case"]["T"], s["case"]["H"])
    moe.rms_norm_bwd(s["dy"], s["total"], s["rstd"], s["weight"], s["dx"], dweight=s["dweight"],
                     d_total=s.get("d_total"), ws=s["ws"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_mx(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    if "w_back" not in s:
        s["w_back"] = torch.empty((c["E"], c["K"], c["N"]), device="cuda", dtype=_dtype(c))
        if not c["back_only"]:
            s["codes"], s["scales"] = moe.mx_alloc(c["E"], c["K"], c["N"])
    if not c["back_only"]:
        moe.mx_quantize(s["w"], s["codes"], s["scales"])
    moe.mx_dequantize(s["codes"], s["scales"], s["w_back"])
    if c["back_only"]:
        return {"w": s["w_back"]}
    return {"w": s["w_back"], "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _own_clip(s):
    import dispatch_gemm_combine_gb300 as moe
    if "table" not in s:
        s["table"] = moe.grad_table(s["grads"], s["out"])
        s["norm"] = torch.empty(2, device="cuda", dtype=torch.float32)
        s["ws"] = moe.grad_clip_workspace(s["table"])
    moe.grad_clip(s["table"], s["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"][0], "grads": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"few": _own_few, "norm_fwd": _own_norm, "norm_bwd": _own_norm_bwd, "mx": _own_mx,
                "clip": _own_clip}[op](state)
    return {"few": _plain_few, "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd,
            "mx": _plain_mx, "clip": _plain_clip}[op](state)


# ------------------------------------------------------------------ necessary work
def work(case):
    c, op = case, case["op"]
    if op == "few":
        T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
        es = 4 if c["weights"] == "fp32" else 2
        # experts that T tokens with k uniform choices each reach, on average
        touched = E * (1.0 - (1.0 - k / E) ** T)
        per = 3 * H * I * (0.5 + 1 / 32 if c["weights"] == "mx" else es)
        if c["bias"]:
            per += es * (2 * I + H)
        x_bytes = T * H * (1 + 1 / 32 if c["x8"] else es)
        return {"bytes": touched * per + x_bytes + T * k * 8 + T * H * es,
                "flops": 2.0 * T * k * 3 * H * I}
    if op == "mx":
        n, es = c["E"] * c["K"] * c["N"], 4 if c["dtype"] == "fp32" else 2
        if c["back_only"]:
            return {"bytes": n * (0.5 + 1 / 32 + es), "flops": n}
        return {"bytes": n * (2 * es + 1 / 32), "flops": 4 * n}
    if op == "norm_fwd":
        n, es = c["T"] * c["H"], 4 if c["dtype"] == "fp32" else 2
        per = es * (3 if c["residual"] else 1) + (1 + 1 / 32 if c["out8"] else es)
        return {"bytes": n * per + c["H"] * es + (4 * c["T"] if c["train"] else 0), "flops": 5 * n}
    if op == "norm_bwd":
        n, es = c["T"] * c["H"], 4 if c["dtype"] == "fp32" else 2
        return {"bytes": n * es * (4 if c["d_total"] else 3) + 4 * c["T"] + c["H"] * (es + 4),
                "flops": 10 * n}
    n = c["count"] * (c["largest"] + 1) / 2 + 3 * c["E"] * c["H"] * c["I"]
    return {"bytes": 2 * n * (4 if c["dtype"] == "fp32" else 2), "flops": 3 * n}


# ------------------------------------------------------------------ 64 bits
def _exact_scale(v, top):
    """The smallest 2^q (q in [-127, 127]) with max |v| <= top * 2^q, last axis."""
    amax = v.abs().amax(-1)
    q = torch.ceil(torch.log2(amax / top))
    q = torch.where(top * torch.exp2(q - 1) >= amax, q - 1, q)
    q = torch.where(top * torch.exp2(q) < amax, q + 1, q)
    return torch.exp2(torch.where(amax == 0, torch.full_like(q, -127.0), q.clamp(-127, 127)))


def _exact_e2m1(code):
    """Values of e2m1 codes from their sign, exponent and mantissa bits."""
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    return torch.where(code >= 8, -mag, mag)


def _exact_mx(codes, scales):
    v = torch.empty((*codes.shape, 2), dtype=torch.float64, device=codes.device)
    v[..., 0], v[..., 1] = _exact_e2m1(codes % 16), _exact_e2m1(codes // 16)
    s = torch.exp2(scales.double() - 127)
    return v.view(*codes.shape[:-1], -1) * s.repeat_interleave(32, -1)


def exact(case, seed):
    if case["op"] == "few" and case["T"] * case["k"] * case["H"] * case["I"] > 6e9:
        return None
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "few":
        x = s["x"].view(torch.float8_e4m3fn).double() if c["x8"] else s["x"].double()
        if c["x8"]:
            x = x * torch.exp2(s["x_scale"].double() - 127).repeat_interleave(32, -1)
        rows = []
        for t in range(c["T"]):
            y = torch.zeros(c["H"], dtype=torch.float64, device="cuda")
            for j, e in enumerate(s["idx"][t].tolist()):
                if c["weights"] == "mx":
                    wgu = _exact_mx(s["mx"][0][e], s["mx"][1][e]).t()
                    wd = _exact_mx(s["mx"][2][e], s["mx"][3][e]).t()
                else:
                    wgu, wd = s["w_gate_up"][e].double(), s["w_down"][e].double()
                h = x[t] @ wgu
                if c["bias"]:
                    h = h + s["b_gate_up"][e].double()
                gate, up = h.view(-1, 2).t() if c["interleaved"] else h.view(2, -1)
                if c["act"] == CLAMPED:
                    gate = torch.minimum(gate, torch.tensor(7.0, dtype=torch.float64, device="cuda"))
                    a = (1 + up.clamp(-7, 7)) * gate / (1 + torch.exp(-1.702 * gate))
                else:
                    a = up * gate / (1 + torch.exp(-gate))
                o = a @ wd
                if c["bias"]:
                    o = o + s["b_down"][e].double()
                y += s["w"][t, j].double() * o
            rows.append(y)
        return {"y": torch.stack(rows)}
    if op == "mx":
        if c["back_only"]:
            return {"w": _exact_mx(s["codes"], s["scales"]).transpose(1, 2)}
        w = s["w"].double().view(c["E"], c["K"] // 32, 32, c["N"]).transpose(2, 3)
        scale = _exact_scale(w, 6.0)[..., None]
        v = w / scale
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1)
        v = (torch.round(v / unit) * unit).clamp(-6, 6) * scale
        return {"w": v.transpose(2, 3).reshape(c["E"], c["K"], c["N"]),
                "scales": scale[..., 0].transpose(1, 2)}
    if op == "norm_fwd":
        r = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        rstd = 1 / torch.sqrt((r * r).sum(-1) / c["H"] + 1e-6)
        y = r * rstd[:, None] * s["weight"].double()
        out = {"y": y}
        if c["out8"]:
            b = y.view(c["T"], -1, 32)
            scale = _exact_scale(b, 448.0)
            out["y"], out["y_scale"] = (b / scale[..., None]).view(c["T"], -1), scale
        if c["residual"]:
            out["total"] = r
        if c["train"]:
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":
        r, dy, w = s["total"].double(), s["dy"].double(), s["weight"].double()
        rstd = s["rstd"].double()[:, None]
        dot = (dy * w * r).sum(-1, keepdim=True)
        dx = rstd * dy * w - r * rstd ** 3 * dot / c["H"]
        if c["d_total"]:
            dx = dx + s["d_total"].double()
        return {"dx": dx, "dweight": (dy * r * rstd).sum(0)}
    norm = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in s["grads"]))
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor(norm, dtype=torch.float64),
            "grads": [t.double() * coef for t in s["grads"]]}
