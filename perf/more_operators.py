"""Cases for the operators of a training step around the expert layer, and their
plain forms.

Three operators are measured, as a transformer block with an expert layer uses
them between its layers, behind its router and before its update:

  join_fwd, join_bwd   a block's output joins the residual stream: the norm after
                       the block (or a weight per column), a gate per token, the
                       scaled residual, and the norm before the next block, with
                       its output in the storage type or as e4m3 with one
                       power-of-two scale per 32 columns; and the gradients
  route_bwd            the router's gradient: through the softmax of the chosen
                       logits, with the load-balancing loss and the z-loss
  orth                 weight updates made orthogonal by Newton-Schulz products

`run` computes a case in elementary torch operations (own = False) or calls
dispatch_gemm_combine_gb300 (own = True).  `exact` computes it in 64 bits.

  join    p = y * rs(y) * post_weight  (post_norm)  or  y * post_weight
          total = residual_scale * residual + gate * p
          n = total * rs(total) * weight,  rs(v) = (mean v^2 + eps)^-1/2
  route   balance = sum_e f_e mean_t softmax(logits)_te,  f_e = counts_e E / (T k)
          z = mean_t (log sum_e exp logits_te)^2
  orth    x_0 = g / (|g|_F + eps),  a = x x^T,  x <- (c0 + c1 a + c2 a^2) x
"""

import math

import torch

own = False

EPS = 1e-6
COEFS = (3.4445, -4.7750, 2.0315)
ORTH_EPS = 1e-7


# ------------------------------------------------------------------ cases
def _join(name, T, H, dtype, post_norm=True, post_weight=True, gate=True, scale=1.0, out="same"):
    """out: the next norm's output, in the storage type ("same"), as "e4m3", or none ("")."""
    return {"name": name, "op": "join_fwd", "T": T, "H": H, "dtype": dtype, "post_norm": post_norm,
            "post_weight": post_weight, "gate": gate, "scale": scale, "out": out}


def _join_bwd(name, T, H, dtype, post_norm=True, post_weight=True, gate=True, scale=1.0, next_norm=True):
    return {"name": name, "op": "join_bwd", "T": T, "H": H, "dtype": dtype, "post_norm": post_norm,
            "post_weight": post_weight, "gate": gate, "scale": scale, "next_norm": next_norm}


def _route(name, T, E, k, balance, z, weights=True):
    return {"name": name, "op": "route_bwd", "T": T, "E": E, "k": k, "balance": balance, "z": z,
            "weights": weights}


def _orth(name, E, M, N, dtype, split=False, steps=5):
    """split: the gate and the up columns of [E, M, N] apart, as strided views."""
    return {"name": name, "op": "orth", "E": E, "M": M, "N": N, "dtype": dtype, "split": split,
            "steps": steps}


def listed():
    return [
        # one decoded token between two blocks of width 2880
        _join("join_one", 1, 2880, "bf16"),
        # a long prompt through a gated block, handed to the next expert layer in 8 bits
        _join("join_long_e4m3", 16384, 4096, "bf16", out="e4m3"),
        # single precision, a weight per column instead of the norm, a scaled residual, ragged sizes
        _join("join_scaled_fp32", 777, 1032, "fp32", post_norm=False, gate=False, scale=1.5),
        # the training backward at the benchmark's size
        _join_bwd("join_bwd_train", 8192, 2880, "bf16"),
        # the last block's backward, where no norm follows: single precision, ragged
        _join_bwd("join_bwd_last_fp32", 1001, 1400, "fp32", gate=False, scale=0.5, next_norm=False),
        # the router of the layer with 128 experts, top-4, at the benchmark's size
        _route("route_bwd_train", 8192, 128, 4, 0.01, 0.001),
        # many tokens over 256 experts, top-8
        _route("route_bwd_many", 65536, 256, 8, 0.001, 0.0),
        # an odd number of experts and few tokens: latency
        _route("route_bwd_small", 37, 61, 6, 0.02, 0.001),
        # the down weights of the tiny single-precision layer (8 experts): latency
        _orth("orth_tiny", 8, 128, 128, "fp32"),
        # the router's weight of a layer with H = 2880 and 128 experts: tall, one matrix
        _orth("orth_router", 1, 2880, 128, "fp32"),
        # ragged bf16 updates, wider than tall
        _orth("orth_ragged", 6, 333, 1001, "bf16"),
        # the gate_up gradients of 4 experts of the H = I = 2880 layer, gate and up apart
        _orth("orth_gate_up", 4, 2880, 5760, "fp32", split=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join_fwd", "join_fwd", "join_bwd", "join_bwd", "route_bwd", "orth", "orth", "orth"])
    if op in ("join_fwd", "join_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        out = rng.choice(["same", "same", "e4m3", ""])
        step = 32 if out == "e4m3" and op == "join_fwd" else 8
        H = step * max(1, _log(rng, 64, 8192) // step)
        T = min(_log(rng, 1, 16384), 16384 * 2048 // H)
        post_norm = rng.random() < 0.7
        args = (T, H, dtype, post_norm, rng.random() < 0.8, rng.random() < 0.5, rng.choice([1.0, 1.0, 0.5, 1.5]))
        c = _join("", *args, out) if op == "join_fwd" else _join_bwd("", *args, rng.random() < 0.7)
    elif op == "route_bwd":
        E = _log(rng, 4, 1024)
        c = _route("", min(_log(rng, 1, 65536), 65536 * 256 // E), E, min(E, rng.choice([1, 2, 4, 6, 8])),
                   rng.choice([0.0, 0.01, 0.1]), rng.choice([0.0, 0.001]), rng.random() < 0.8)
        if not (c["balance"] or c["z"]):
            c["weights"] = True
    else:
        M, N = _log(rng, 16, 2880), _log(rng, 16, 2880)
        m, n = min(M, N), max(M, N)
        E = min(_log(rng, 1, 32), max(1, int(8e10 / (m * m * n))))
        split = rng.random() < 0.25
        c = _orth("", E, M, 2 * N if split else N, rng.choice(["fp32", "bf16"]), split, rng.choice([5, 5, 5, 3]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _randn(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, s = case, {"case": case}
    if c["op"] in ("join_fwd", "join_bwd"):
        T, H, dt = c["T"], c["H"], _dtype(c)
        # a block's output, of a size that grows over the columns, and the residual stream
        s["y"] = (_randn(g, (T, H)) * torch.linspace(0.3, 1.5, H, device="cuda")).to(dt)
        s["post_weight"] = (1 + _randn(g, (H,), 0.1)).to(dt) if c["post_weight"] else None
        s["gate"] = torch.sigmoid(_randn(g, (T,))) if c["gate"] else None
        s["weight"] = (1 + _randn(g, (H,), 0.1)).to(dt)
        residual = _randn(g, (T, H), 3.0).to(dt)
        if c["op"] == "join_fwd":
            s["residual"] = residual
            return s
        # what the forward left for the backward
        p, rs_y = _post(c, s, torch.float64)
        total = c["scale"] * residual.double() + (p * s["gate"].double()[:, None] if c["gate"] else p)
        s["total"] = total.to(dt)
        s["rstd_post"] = rs_y[:, 0].float() if c["post_norm"] else None
        s["dn"] = s["rstd"] = None
        if c["next_norm"]:
            s["rstd"] = torch.rsqrt(total.square().mean(-1) + EPS).float()
            s["dn"] = _randn(g, (T, H)).to(dt)
        else:
            s["weight"] = None
        s["d_total"] = _randn(g, (T, H)).to(dt)
    elif c["op"] == "route_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        # a router with some experts in favour
        s["logits"] = _randn(g, (T, E), 1.5) + _randn(g, (E,), 0.7)
        top = torch.topk(s["logits"], k, dim=-1)
        s["idx"] = top.indices.to(torch.int32).contiguous()
        s["w"] = torch.softmax(top.values, dim=-1)
        s["counts"] = torch.bincount(s["idx"].flatten().long(), minlength=E).to(torch.int32)
        s["dw"] = _randn(g, (T, k), 0.05) if c["weights"] else None
    else:
        E, M, N, dt = c["E"], c["M"], c["N"], _dtype(c)
        # gradients whose rows and columns differ in size
        w = _randn(g, (E, M, N), 0.01)
        w *= torch.exp(0.5 * _randn(g, (E, M, 1)))
        w *= torch.exp(0.5 * _randn(g, (E, 1, N)))
        if E >= 6:
            w[E - 1] = 0          # an expert that no token has reached yet
        s["g"] = w.to(dt)
    return s


# ------------------------------------------------------------------ plain forms
def _post(c, s, wide):
    """The block's output as it joins (before the gate), and its 1 / rms, in `wide`."""
    y = s["y"].to(wide)
    rs = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    p = y * rs if c["post_norm"] else y
    return (p * s["post_weight"].to(wide) if c["post_weight"] else p), rs


def _to_e4m3(v):
    """(codes as float8_e4m3fn, scale bytes) of v [T, H]: per 32 columns the smallest
    power of two 2^q (q in [-127, 127]) with amax <= 448 * 2^q; the byte is q + 127."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    frac, exp = torch.frexp(amax)
    q = exp.to(torch.int32) - 9 + (frac > 0.875).to(torch.int32)
    q = torch.where(amax == 0, torch.full_like(q, -127), q.clamp(-127, 127))
    code = torch.ldexp(b, -q[..., None]).float().to(torch.float8_e4m3fn)
    return code.reshape(v.shape), (q + 127).to(torch.uint8)


def _plain_join(s):
    c, dt = s["case"], _dtype(s["case"])
    # the 8-bit output rounds and scales by borders: 64 bits up to there
    wide = torch.float64 if c["out"] == "e4m3" else torch.float32
    p, rs_y = _post(c, s, wide)
    if c["gate"]:
        p = p * s["gate"].to(wide)[:, None]
    total = c["scale"] * s["residual"].to(wide) + p
    out = {"total": total.to(dt)}
    if c["post_norm"]:
        out["rstd_post"] = rs_y[:, 0].float()
    if c["out"]:
        rs = torch.rsqrt(total.square().mean(-1, keepdim=True) + EPS)
        n = total * rs * s["weight"].to(wide)
        out["rstd"] = rs[:, 0].float()
        if c["out"] == "e4m3":
            out["n"], byte = _to_e4m3(n)
            out["n_scale"] = byte.view(torch.float8_e8m0fnu)
        else:
            out["n"] = n.to(dt)
    return out


def _plain_join_bwd(s):
    c, dt = s["case"], _dtype(s["case"])
    dr = s["d_total"].float()
    out = {}
    if c["next_norm"]:
        rhat = s["total"].float() * s["rstd"][:, None]
        dn = s["dn"].float()
        dnw = dn * s["weight"].float()
        dr = dr + s["rstd"][:, None] * (dnw - rhat * (dnw * rhat).mean(-1, keepdim=True))
        out["d_weight"] = (dn * rhat).double().sum(0).float()
    y = s["y"].float()
    yhat = y * s["rstd_post"][:, None] if c["post_norm"] else y
    w = s["post_weight"].float() if c["post_weight"] else torch.ones(c["H"], device=y.device)
    dp = dr * s["gate"][:, None] if c["gate"] else dr
    if c["gate"]:
        out["d_gate"] = (dr * yhat * w).double().sum(-1).float()
    if c["post_weight"]:
        out["d_post_weight"] = (dp * yhat).double().sum(0).float()
    dy = dp * w
    if c["post_norm"]:
        dy = s["rstd_post"][:, None] * (dy - yhat * (dy * yhat).mean(-1, keepdim=True))
    out["dy"] = dy.to(dt)
    out["d_residual"] = (c["scale"] * dr).to(dt)
    return out


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    v = s["logits"]
    top = v.amax(-1, keepdim=True)
    e = torch.exp(v - top)
    sums = e.sum(-1, keepdim=True)
    p, lse = e / sums, top + torch.log(sums)
    f = s["counts"].float() * (E / (T * k))
    fp = (p * f).sum(-1, keepdim=True)
    d = (c["balance"] / T) * p * (f - fp) + (2 * c["z"] / T) * lse * p
    if c["weights"]:
        w, dw = s["w"], s["dw"]
        d.scatter_add_(1, s["idx"].long(), w * (dw - (w * dw).sum(-1, keepdim=True)))
    losses = torch.stack((fp.double().mean(), lse.double().square().mean())).float()
    return {"d_logits": d, "losses": losses}


def _plain_orth_one(g, steps):
    flip = g.shape[1] > g.shape[2]
    x = g.float().transpose(1, 2) if flip else g.float()
    x = x / (torch.sqrt(x.square().sum((1, 2), keepdim=True)) + ORTH_EPS)
    for _ in range(steps):
        a = x @ x.transpose(1, 2)
        x = COEFS[0] * x + (COEFS[1] * a + COEFS[2] * (a @ a)) @ x
    return (x.transpose(1, 2) if flip else x).to(torch.bfloat16).contiguous()


def _views(c, t):
    """The matrices of [E, M, N] that are made orthogonal: all of it, or its halves."""
    return t.split(c["N"] // 2, dim=2) if c["split"] else (t,)


def _plain_orth(s):
    c = s["case"]
    return {"out": torch.cat([_plain_orth_one(g, c["steps"]) for g in _views(c, s["g"])], dim=2)}


# ------------------------------------------------------------------ the framework's operators
def _own_join(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    T, H, dt = c["T"], c["H"], _dtype(c)
    if "total" not in s:      # what a program keeps between calls
        s["total"] = torch.empty((T, H), device="cuda", dtype=dt)
        s["rs_y"] = torch.empty(T, device="cuda") if c["post_norm"] else None
        s["rs"] = torch.empty(T, device="cuda") if c["out"] else None
        e4m3 = c["out"] == "e4m3"
        s["n"] = torch.empty((T, H), device="cuda", dtype=torch.float8_e4m3fn if e4m3 else dt) if c["out"] else None
        s["n_scale"] = torch.empty((T, H // 32), device="cuda", dtype=torch.uint8) if e4m3 else None
    moe.join_norm_fwd(s["y"], s["residual"], s["total"], post_norm=c["post_norm"],
                      post_weight=s["post_weight"], gate=s["gate"], residual_scale=c["scale"],
                      weight=s["weight"] if c["out"] else None, n=s["n"], n_scale=s["n_scale"], eps=EPS,
                      rstd_post=s["rs_y"], rstd=s["rs"])
    out = {"total": s["total"]}
    if c["post_norm"]:
        out["rstd_post"] = s["rs_y"]
    if c["out"]:
        out["rstd"], out["n"] = s["rs"], s["n"]
    if c["out"] == "e4m3":
        out["n_scale"] = s["n_scale"].view(torch.float8_e8m0fnu)
    return out


def _own_join_bwd(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    T, H = c["T"], c["H"]
    if "dy" not in s:
        s["dy"], s["d_residual"] = torch.empty_like(s["y"]), torch.empty_like(s["y"])
        s["d_gate"] = torch.empty(T, device="cuda") if c["gate"] else None
        s["d_post_weight"] = torch.empty(H, device="cuda") if c["post_weight"] else None
        s["d_weight"] = torch.empty(H, device="cuda") if c["next_norm"] else None
        s["ws"] = moe.join_norm_workspace(T, H)
    moe.join_norm_bwd(s["y"], s["dy"], s["d_residual"], d_total=s["d_total"], dn=s["dn"], total=s["total"],
                      weight=s["weight"], rstd=s["rstd"], post_norm=c["post_norm"],
                      post_weight=s["post_weight"], rstd_post=s["rstd_post"], gate=s["gate"],
                      residual_scale=c["scale"], d_gate=s["d_gate"], d_post_weight=s["d_post_weight"],
                      d_weight=s["d_weight"], ws=s["ws"])
    out = {n: s[n] for n in ("d_weight", "d_gate", "d_post_weight") if s[n] is not None}
    out["dy"], out["d_residual"] = s["dy"], s["d_residual"]
    return out


def _own_route(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    if "shape" not in s:
        s["shape"] = moe.Shape(c["T"], 8, 8, c["E"], c["k"])
        s["ws"] = moe.route_bwd_workspace(s["shape"])
        s["d_logits"] = torch.empty((c["T"], c["E"]), device="cuda")
        s["losses"] = torch.empty(2, device="cuda")
    moe.route_bwd(s["shape"], s["logits"], s["d_logits"], s["ws"], topk_idx=s["idx"], topk_w=s["w"],
                  d_topk_w=s["dw"], counts=s["counts"], balance=c["balance"], z=c["z"], losses=s["losses"])
    return {"d_logits": s["d_logits"], "losses": s["losses"]}


def _own_orth(s):
    import dispatch_gemm_combine_gb300 as moe
    c = s["case"]
    if "out" not in s:
        s["out"] = torch.empty((c["E"], c["M"], c["N"]), device="cuda", dtype=torch.bfloat16)
        s["ws"] = moe.orthogonalize_workspace(_views(c, s["g"])[0])
    for g, out in zip(_views(c, s["g"]), _views(c, s["out"])):
        moe.orthogonalize(g, out, s["ws"], steps=c["steps"], coefs=COEFS, eps=ORTH_EPS)
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"join_fwd": _own_join, "join_bwd": _own_join_bwd, "route_bwd": _own_route,
                "orth": _own_orth}[op](state)
    return {"join_fwd": _plain_join, "join_bwd": _plain_join_bwd, "route_bwd": _plain_route,
            "orth": _plain_orth}[op](state)


# ------------------------------------------------------------------ necessary work
def work(case):
    c, op = case, case["op"]
    if op in ("join_fwd", "join_bwd"):
        T, H, es = c["T"], c["H"], 4 if c["dtype"] == "fp32" else 2
        rows = 4 * T * ((1 if c["gate"] else 0) + (1 if c["post_norm"] else 0))
        if op == "join_fwd":
            per = 3 * es + {"": 0, "same": es, "e4m3": 1 + 1 / 32}[c["out"]]
            rows += 4 * T if c["out"] else 0
            cols = H * es * ((1 if c["post_weight"] else 0) + (1 if c["out"] else 0))
            return {"bytes": T * H * per + rows + cols, "flops": 12 * T * H}
        per = es * (4 + (2 if c["next_norm"] else 0))     # d_total, y, dy, d_residual; dn, total
        rows += 4 * T * ((1 if c["gate"] else 0) + (1 if c["next_norm"] else 0))
        cols = H * (es + 4) * ((1 if c["post_weight"] else 0) + (1 if c["next_norm"] else 0))
        return {"bytes": T * H * per + rows + cols, "flops": 24 * T * H}
    if op == "route_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 8 * T * E + (12 * T * k if c["weights"] else 0) + 4 * E + 8, "flops": 10 * T * E}
    m, n = sorted((c["M"], c["N"] // (2 if c["split"] else 1)))
    batch = c["E"] * (2 if c["split"] else 1)
    # a = x x^T and a a are symmetric: half of their products
    return {"bytes": batch * m * n * (2 + (4 if c["dtype"] == "fp32" else 2)),
            "flops": batch * c["steps"] * (m * m * n + m ** 3 + 2 * m * m * n)}


# ------------------------------------------------------------------ 64 bits
def _exact_join(c, s):
    y = s["y"].double()
    H = c["H"]
    out = {}
    p = y
    if c["post_norm"]:
        rs = 1 / torch.sqrt((y * y).sum(-1) / H + EPS)
        out["rstd_post"] = rs
        p = p * rs[:, None]
    if c["post_weight"]:
        p = p * s["post_weight"].double()
    if c["gate"]:
        p = s["gate"].double()[:, None] * p
    total = s["residual"].double() * c["scale"] + p
    res = {"total": total, **out}
    if c["out"]:
        rs = 1 / torch.sqrt((total * total).sum(-1) / H + EPS)
        res["rstd"] = rs
        n = total * rs[:, None] * s["weight"].double()
        res["n"] = n
        if c["out"] == "e4m3":
            b = n.view(c["T"], -1, 32)
            amax = b.abs().amax(-1)
            q = torch.ceil(torch.log2(amax / 448))
            q = torch.where(448 * torch.exp2(q - 1) >= amax, q - 1, q)
            q = torch.where(448 * torch.exp2(q) < amax, q + 1, q)
            scale = torch.exp2(torch.where(amax == 0, torch.full_like(q, -127.0), q.clamp(-127, 127)))
            res["n"], res["n_scale"] = (b / scale[..., None]).view(c["T"], -1), scale
    return res


def _exact_join_bwd(c, s):
    """Through the next norm by its formula (total and its 1 / rms are given, each as
    rounded), through the rest by differentiation."""
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    dr, res = s["d_total"].double(), {}
    if c["next_norm"]:
        r, rs, dn = s["total"].double(), s["rstd"].double()[:, None], s["dn"].double()
        dnw = dn * s["weight"].double()
        dr = dr + rs * dnw - r * rs ** 3 * (dnw * r).sum(-1, keepdim=True) / c["H"]
        res["d_weight"] = torch.einsum("th,th->h", dn, r * rs)
    y, gate = leaf(s["y"]), leaf(s["gate"] if c["gate"] else torch.ones(c["T"], device="cuda"))
    w = leaf(s["post_weight"] if c["post_weight"] else torch.ones(c["H"], device="cuda"))
    p = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["H"] + EPS) if c["post_norm"] else y
    dy, d_gate, dw = torch.autograd.grad((dr * (gate[:, None] * (p * w))).sum(), (y, gate, w))
    if c["gate"]:
        res["d_gate"] = d_gate
    if c["post_weight"]:
        res["d_post_weight"] = dw
    res["dy"], res["d_residual"] = dy, dr * c["scale"]
    return res


def _exact_route(c, s):
    """By differentiation of the losses."""
    v = s["logits"].double().requires_grad_()
    f = s["counts"].double() * c["E"] / (c["T"] * c["k"])
    balance = (torch.softmax(v, dim=-1).mean(0) * f).sum()
    z = torch.logsumexp(v, dim=-1).square().mean()
    loss = c["balance"] * balance + c["z"] * z
    if c["weights"]:
        # the weights are given, as rounded; their derivative is w_i (1[i = j] - w_j)
        chosen = v.gather(1, s["idx"].long())
        w, dw = s["w"].double(), s["dw"].double()
        loss = loss + (chosen * (w * dw - w * (w * dw).sum(-1, keepdim=True))).sum()
    d = torch.autograd.grad(loss, v)[0]
    return {"d_logits": d, "losses": torch.stack((balance, z)).detach()}


def exact(case, seed):
    c = case
    if c["op"] == "orth":
        m, n = sorted((c["M"], c["N"] // (2 if c["split"] else 1)))
        if c["E"] * (2 if c["split"] else 1) * c["steps"] * m * m * n * 6.0 > 8e12:
            return None
    s = prepare(case, seed)
    if c["op"] == "join_fwd":
        return _exact_join(c, s)
    if c["op"] == "join_bwd":
        return _exact_join_bwd(c, s)
    if c["op"] == "route_bwd":
        return _exact_route(c, s)
    out = torch.empty((c["E"], c["M"], c["N"]), dtype=torch.float64, device="cuda")
    for g, o in zip(_views(c, s["g"]), _views(c, out)):
        for e in range(c["E"]):
            x = g[e].double()
            x = x / (torch.linalg.vector_norm(x) + ORTH_EPS)
            for _ in range(c["steps"]):
                # x (c0 + c1 b + c2 b^2) with b = x^T x, from the narrower side
                if x.shape[0] <= x.shape[1]:
                    b1 = x @ x.t() @ x
                    b2 = x @ x.t() @ b1
                else:
                    b1 = x @ (x.t() @ x)
                    b2 = b1 @ (x.t() @ x)
                x = COEFS[0] * x + COEFS[1] * b1 + COEFS[2] * b2
            o[e] = x
    return {"out": out}
