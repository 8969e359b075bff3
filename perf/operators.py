"""The operators around the FP8 linear: cases, plain forms and the library's calls.

* norm      -- root-mean-square norm with the residual's addition and FP8 codes out
               (one delayed scale per tensor, or one current scale per row)
* norm_grad -- its gradient: dx with the residual stream's gradient, dgamma
* mm        -- FP8 product with scale, bias, activation and a residual (added) or gate
               (multiplied) operand in its epilogue; bf16 out, or FP8 codes with a ring
* act_grad  -- the gradient of that epilogue, cast to FP8 for the backward products,
               with the bias gradients

``run`` computes an operator in its plain form, or with ``own`` set by the calls of
``fp8_delayed_scaling_02_b200.ops``.  FP8 codes are returned as the values they stand for.
"""

import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
GELU_C = 0.7978845608028654  # sqrt(2 / pi)
GELU_A = 0.044715


def listed():
    return [
        # One token of a decode step: latency; a row scale keeps serving free of state.
        dict(name="norm_one_token", op="norm", rows=1, cols=1536, dtype="bf16", residual=True, scale="row", fmt="e4m3"),
        # The norm before a linear of the 1.2B model, training: 8192 tokens, delayed scaling.
        dict(name="norm_train", op="norm", rows=8192, cols=1536, dtype="bf16", residual=True, scale="ring", fmt="e4m3"),
        # Rows of an odd width, whose vectors start at every alignment.
        dict(name="norm_ragged", op="norm", rows=1000, cols=1537, dtype="fp16", residual=False, scale="ring",
             fmt="e4m3"),
        # The gradient of norm_train, joined with the residual stream's.
        dict(name="norm_grad_train", op="norm_grad", rows=8192, cols=1536, dtype="bf16", dres=True),
        # A float32 stream, FFN-wide rows: a norm inside the feed-forward.
        dict(name="norm_grad_wide", op="norm_grad", rows=2048, cols=4096, dtype="fp32", dres=False),
        # The gate product of one decoded token: reading the weight is all there is.
        dict(name="mm_one_token", op="mm", M=1, N=4096, K=1536, act="silu", aux="mul", bias=False, z=False, out="bf16",
             scale="row"),
        # The gate product of the 1.2B model, training: pre-activation kept for the
        # backward, gated, cast for the next product.
        dict(name="mm_gate_train", op="mm", M=8192, N=4096, K=1536, act="silu", aux="mul", bias=False, z=True,
             out="e4m3", scale="tensor"),
        # The product that closes the feed-forward, added to the residual stream.
        dict(name="mm_down_train", op="mm", M=8192, N=1536, K=4096, act="none", aux="add", bias=False, z=False,
             out="bf16", scale="tensor"),
        # An odd number of outputs, with a bias: rows whose stores start at every alignment.
        dict(name="mm_ragged", op="mm", M=1000, N=1537, K=2048, act="gelu", aux="none", bias=True, z=True, out="e4m3",
             scale="tensor"),
        # The gradient of mm_gate_train's epilogue.
        dict(name="act_grad_gated", op="act_grad", rows=8192, cols=4096, dtype="bf16", act="silu", gate=True, db=False),
        # A short batch with bias gradients.
        dict(name="act_grad_bias", op="act_grad", rows=512, cols=4096, dtype="bf16", act="gelu", gate=False, db=True),
        # Odd rows, float32 gradient.
        dict(name="act_grad_ragged", op="act_grad", rows=1000, cols=1537, dtype="fp32", act="relu", gate=False,
             db=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Rows of one token to 16384, widths of 64 to 8192 (odd ones among them); the largest
    tensor and the largest product are those of the listed cases."""
    op = rng.choice(["norm", "norm_grad", "mm", "act_grad"])
    most = 8192 * 4096
    if op == "mm":
        K = 16 * _log(rng, 8, 256)
        N = _log(rng, 64, 8192)
        N = N if rng.random() < 0.3 else max(64, N // 16 * 16)
        M = _log(rng, 1, max(1, min(8192, most * 1536 // (N * K), most // N)))
        out = rng.choice(["bf16", "e4m3"])
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "relu", "gelu", "silu"]),
                    aux=rng.choice(["none", "add", "mul"]), bias=rng.random() < 0.5, z=rng.random() < 0.5, out=out,
                    scale=rng.choice(["tensor", "row"]))
    cols = _log(rng, 64, 8192)
    cols = cols if rng.random() < 0.3 else max(64, cols // 8 * 8)
    rows = _log(rng, 1, max(1, min(16384, most // (2 * cols))))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7,
                    scale=rng.choice(["ring", "row"]), fmt="e4m3")
    if op == "norm_grad":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, dres=rng.random() < 0.7)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, act=rng.choice(["relu", "gelu", "silu"]),
                gate=rng.random() < 0.5, db=rng.random() < 0.5)


def _normal(g, shape, std=1.0, outliers=False):
    v = torch.randn(shape, generator=g, device="cuda") * std
    if outliers:  # 0.5% of the entries are 30 times as large, as activations have them
        v = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.005, v * 30.0, v)
    return v


def _ring(g, fmt, amax):
    """A ring in mid-training: sixteen earlier amaxes near `amax`, the scale they give."""
    hist = amax * (0.8 + 0.4 * torch.rand(16, generator=g, device="cuda"))
    scale = (FMAX[fmt] / hist.max()).reshape(1)
    idx = torch.randint(0, 16, (1,), generator=g, device="cuda", dtype=torch.int32)
    if own:
        from fp8_delayed_scaling_02_b200 import ops
        r = ops.Ring("cuda")
        r.history.copy_(hist)
        r.idx.copy_(idx)
        r.scale.copy_(scale)
        return r
    return dict(history=hist, idx=idx, scale=scale, scale_inv=torch.ones_like(scale))


def _codes(v, fmt, per_row):
    """FP8 codes of v (their bytes) and the factor that undoes their scale."""
    amax = v.abs().amax(dim=1) if per_row else v.abs().max().reshape(1)
    s = FMAX[fmt] / amax
    q = (v * (s[:, None] if per_row else s)).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    return q.view(torch.uint8), 1.0 / s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    s = dict(case)
    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        s["a"], s["sinv_a"] = _codes(_normal(g, (M, K), 1.0, True), "e4m3", c["scale"] == "row")
        s["b"], s["sinv_b"] = _codes(_normal(g, (N, K), 0.02), "e4m3", False)
        s["bias_v"] = _normal(g, (N,), 0.5) if c["bias"] else None
        s["aux_v"] = _normal(g, (M, N)).to(torch.bfloat16) if c["aux"] != "none" else None
        s["ring"] = _ring(g, "e4m3", 30.0) if c["out"] == "e4m3" else None
        return s
    rows, cols, dt = c["rows"], c["cols"], DT[c["dtype"]]
    if c["op"] == "norm":
        s["x"] = _normal(g, (rows, cols), 1.0, True).to(dt)
        s["res"] = _normal(g, (rows, cols)).to(dt) if c["residual"] else None
        s["gamma"] = (1.0 + _normal(g, (cols,), 0.1)).to(dt)
        s["ring"] = _ring(g, c["fmt"], 60.0) if c["scale"] == "ring" else None
    elif c["op"] == "norm_grad":
        h = _normal(g, (rows, cols), 1.5, True).to(dt)
        s["h"] = h
        s["rstd"] = torch.rsqrt(h.double().square().mean(dim=1) + EPS).float()
        s["gamma"] = (1.0 + _normal(g, (cols,), 0.1)).to(dt)
        s["dy"] = _normal(g, (rows, cols), 1e-3).to(dt)
        s["dres_v"] = _normal(g, (rows, cols), 1e-3).to(dt) if c["dres"] else None
    else:
        s["dy"] = _normal(g, (rows, cols), 1e-3).to(dt)
        s["zv"] = _normal(g, (rows, cols), 1.5).to(torch.bfloat16)
        s["u"] = _normal(g, (rows, cols)).to(torch.bfloat16) if c["gate"] else None
        s["ring"] = _ring(g, "e5m2", 8e-3)
        s["ring_u"] = _ring(g, "e5m2", 1.5e-2) if c["gate"] else None
    return s


# ---- plain forms ------------------------------------------------------------------


def _fold(ring, amax, fmt):
    """The ring after a call whose tensor has this amax."""
    s = ring["scale"].clone()
    ring["history"].index_copy_(0, ring["idx"].long(), amax.reshape(1))
    ring["idx"].copy_((ring["idx"] + 1) % 16)
    m = ring["history"].max()
    new = FMAX[fmt] / m
    ring["scale"].copy_(torch.where((m > 0) & torch.isfinite(m) & torch.isfinite(new), new, s))
    ring["scale_inv"].copy_(1.0 / s)


def _cast(v, scale, fmt):
    return (v * scale).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _ring_out(ring):
    if isinstance(ring, dict):
        return dict(ring)
    return dict(history=ring.history, idx=ring.idx, scale=ring.scale, scale_inv=ring.scale_inv)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z / (1.0 + torch.exp(-2.0 * GELU_C * (z + GELU_A * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    p = 1.0 / (1.0 + torch.exp(-2.0 * GELU_C * (z + GELU_A * z * z * z)))
    return p + z * p * (1.0 - p) * (2.0 * GELU_C) * (1.0 + 3.0 * GELU_A * z * z)


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(s["x"].dtype).float()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)
    y = h * rstd[:, None] * s["gamma"].float()
    out = dict(rstd=rstd)
    if s["res"] is not None:
        out["h"] = h.to(s["x"].dtype)
    if s["ring"] is not None:
        out["codes"] = _cast(y, s["ring"]["scale"], s["fmt"])
        _fold(s["ring"], y.abs().max(), s["fmt"])
        out["ring"] = _ring_out(s["ring"])
    else:
        a = y.abs().amax(dim=1)
        scale = torch.where(a > 0, FMAX[s["fmt"]] / a, torch.ones_like(a))
        out["codes"] = _cast(y, scale[:, None], s["fmt"])
        out["sinv"] = 1.0 / scale
    return out


def _plain_norm_grad(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["dres_v"] is not None:
        dx = dx + s["dres_v"].float()
    return dict(dx=dx.to(s["h"].dtype), dgamma=(dy * xh).sum(dim=0))


def _plain_mm(s):
    a = s["a"].view(F8["e4m3"]).float()
    b = s["b"].view(F8["e4m3"]).float()
    z = (a @ b.t()) * (s["sinv_a"] * s["sinv_b"]).reshape(-1, 1)
    if s["bias_v"] is not None:
        z = z + s["bias_v"]
    y = _act(z, s["act"])
    if s["aux"] != "none":
        y = y * s["aux_v"].float() if s["aux"] == "mul" else y + s["aux_v"].float()
    out = dict(z=z.to(torch.bfloat16)) if s["z"] else {}
    if s["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["y"] = _cast(y, s["ring"]["scale"], "e4m3")
        _fold(s["ring"], y.abs().max(), "e4m3")
        out["ring"] = _ring_out(s["ring"])
    return out


def _plain_act_grad(s):
    dy, z = s["dy"].float(), s["zv"].float()
    dz = dy * _act_slope(z, s["act"])
    out = {}
    if s["u"] is not None:
        dz = dz * s["u"].float()
        du = dy * _act(z, s["act"])
        out["du"] = _cast(du, s["ring_u"]["scale"], "e5m2")
        _fold(s["ring_u"], du.abs().max(), "e5m2")
        out["ring_u"] = _ring_out(s["ring_u"])
        if s["db"]:
            out["dbu"] = du.sum(dim=0)
    out["dz"] = _cast(dz, s["ring"]["scale"], "e5m2")
    _fold(s["ring"], dz.abs().max(), "e5m2")
    out["ring"] = _ring_out(s["ring"])
    if s["db"]:
        out["db"] = dz.sum(dim=0)
    return out


# ---- the library's calls -----------------------------------------------------------


def _own_run(s):
    from fp8_delayed_scaling_02_b200 import ops
    act = {"none": ops.ACT_NONE, "relu": ops.ACT_RELU, "gelu": ops.ACT_GELU, "silu": ops.ACT_SILU}
    if s["op"] == "norm":
        r = ops.rmsnorm(s["x"], s["gamma"], residual=s["res"], eps=EPS, fmt=ops.E4M3, ring=s["ring"], need_rstd=True)
        out = dict(codes=r.codes.view(F8["e4m3"]), rstd=r.rstd)
        if s["res"] is not None:
            out["h"] = r.h
        if s["ring"] is not None:
            out["ring"] = _ring_out(s["ring"])
        else:
            out["sinv"] = r.sinv
        return out
    if s["op"] == "norm_grad":
        dx, dgamma = ops.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["gamma"], dres=s["dres_v"])
        return dict(dx=dx, dgamma=dgamma)
    if s["op"] == "mm":
        y, z = ops.mm_act(s["a"], s["b"], s["sinv_a"], s["sinv_b"], act[s["act"]], bias=s["bias_v"], aux=s["aux_v"],
                          aux_op=ops.AUX_MUL if s["aux"] == "mul" else ops.AUX_ADD, need_z=s["z"],
                          out_fmt=ops.E4M3 if s["out"] == "e4m3" else None, out_ring=s["ring"])
        out = dict(z=z) if s["z"] else {}
        if s["out"] == "bf16":
            out["y"] = y
        else:
            out["y"] = y.view(F8["e4m3"])
            out["ring"] = _ring_out(s["ring"])
        return out
    r = ops.act_backward(s["dy"], s["zv"], act[s["act"]], ops.E5M2, s["ring"], u=s["u"], ring_u=s["ring_u"],
                         need_db=s["db"])
    out = dict(dz=r.dz.view(F8["e5m2"]), ring=_ring_out(s["ring"]))
    if s["db"]:
        out["db"] = r.db
    if s["u"] is not None:
        out["du"] = r.du.view(F8["e5m2"])
        out["ring_u"] = _ring_out(s["ring_u"])
        if s["db"]:
            out["dbu"] = r.dbu
    return out


def run(state):
    if own:
        return _own_run(state)
    return dict(norm=_plain_norm, norm_grad=_plain_norm_grad, mm=_plain_mm, act_grad=_plain_act_grad)[state["op"]](state)


def work(case):
    c = case
    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        b = M * K + N * K + M * N * (2 if c["out"] == "bf16" else 1)
        b += (2 * M * N if c["aux"] != "none" else 0) + (2 * M * N if c["z"] else 0) + (4 * N if c["bias"] else 0)
        return dict(bytes=b + (4 * M if c["scale"] == "row" else 4), flops=2 * M * N * K)
    n, e = c["rows"] * c["cols"], BYTES[c["dtype"]]
    if c["op"] == "norm":
        b = n * e * (3 if c["residual"] else 1) + n + c["cols"] * e + 4 * c["rows"] * (2 if c["scale"] == "row" else 1)
        return dict(bytes=b, flops=6 * n)
    if c["op"] == "norm_grad":
        return dict(bytes=n * e * (4 if c["dres"] else 3) + c["cols"] * (e + 4) + 4 * c["rows"], flops=10 * n)
    b = n * (e + 2 + 1 + (3 if c["gate"] else 0)) + (4 * c["cols"] * (2 if c["gate"] else 1) if c["db"] else 0)
    return dict(bytes=b, flops=12 * n)


# ---- the operators' definitions in 64 bits -------------------------------------------


def _grid(v, fmt):
    """float64 values rounded to the nearest value of the format (ties to even), saturating."""
    mant, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = (torch.frexp(v)[1] - 1).clamp(min=emin) - mant
    step = torch.exp2(e.double())
    return (torch.round(v / step) * step).clamp(-FMAX[fmt], FMAX[fmt])


def _exact_codes(v, ring, fmt):
    """Codes' values of v under the ring's scale, and the ring afterwards."""
    s = ring["scale"].double()
    hist = ring["history"].double().clone()
    hist[int(ring["idx"])] = v.abs().max()
    return _grid(v * s, fmt), dict(history=hist, idx=None, scale=(FMAX[fmt] / hist.max()).reshape(1), scale_inv=1.0 / s)


def _exact_act(z, act):
    """act(z) and its slope, from their definitions by tanh and the logistic function."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    t = torch.tanh(GELU_C * (z + GELU_A * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * z * z)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["x"].dtype).double()  # the stream is kept in its own type
        rstd = (h.pow(2).sum(1) / s["cols"] + EPS).pow(-0.5)
        y = h * s["gamma"].double() * rstd[:, None]
        out = dict(rstd=rstd)
        if s["res"] is not None:
            out["h"] = h
        if s["ring"] is not None:
            out["codes"], out["ring"] = _exact_codes(y, s["ring"], s["fmt"])
        else:
            a = y.abs().max(dim=1).values
            out["sinv"] = a / FMAX[s["fmt"]]
            out["codes"] = _grid(y / out["sinv"][:, None], s["fmt"])
        return out
    if s["op"] == "norm_grad":
        h, r, dy = s["h"].double(), s["rstd"].double()[:, None], s["dy"].double()
        g = dy * s["gamma"].double()
        dx = r * g - h * r ** 3 * (g * h).sum(1, keepdim=True) / s["cols"]
        if s["dres_v"] is not None:
            dx = dx + s["dres_v"].double()
        return dict(dx=dx, dgamma=torch.einsum("rc,rc,r->c", dy, h, r[:, 0]))
    if s["op"] == "mm":
        z = s["a"].view(F8["e4m3"]).double() @ s["b"].view(F8["e4m3"]).double().t()
        z = z * s["sinv_a"].double().reshape(-1, 1) * s["sinv_b"].double()
        if s["bias_v"] is not None:
            z = z + s["bias_v"].double()
        y = _exact_act(z, s["act"])[0]
        if s["aux"] == "add":
            y = y + s["aux_v"].double()
        elif s["aux"] == "mul":
            y = y * s["aux_v"].double()
        out = dict(z=z) if s["z"] else {}
        if s["out"] == "bf16":
            out["y"] = y
        else:
            out["y"], out["ring"] = _exact_codes(y, s["ring"], "e4m3")
        return out
    dy, z = s["dy"].double(), s["zv"].double()
    t, slope = _exact_act(z, s["act"])
    dz = dy * slope * (s["u"].double() if s["u"] is not None else 1.0)
    out = {}
    if s["u"] is not None:
        du = dy * t
        out["du"], out["ring_u"] = _exact_codes(du, s["ring_u"], "e5m2")
        if s["db"]:
            out["dbu"] = du.sum(0)
    out["dz"], out["ring"] = _exact_codes(dz, s["ring"], "e5m2")
    if s["db"]:
        out["db"] = dz.sum(0)
    return out
