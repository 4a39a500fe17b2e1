"""The feed-forward operators' workloads: a transformer block's linear layer,
gated unit and layer norm, forward and backward.

``listed()`` gives the fixed cases, ``draw(rng)`` one more of the same ranges.
``prepare(case, seed)`` makes a case's device tensors, ``run(state)`` is one
pass: the framework's calls where the module's ``own`` is true, and the plain
form otherwise (elementary torch operations in FP32, rounded once at the end).
``exact(case, seed)`` evaluates the definitions in FP64, written apart from
the plain form.  ``work(case)`` counts the bytes and operations that a pass
cannot do without.

Layouts: every matrix is row-major with a leading stride; tokens are rows.

  linear           Y = act(X W^T + bias) + R;  with save: Z = X W^T + bias
  linear_backward  dZ = dY act'(Z);  dX = dZ W,  dW = dZ^T X,  db = sum dZ
  gated            H = act(X Wg^T) * (X Wu^T);  with save: G, U
  gated_backward   dG = dH U act'(G), dU = dH act(G);
                   dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X
  layer_norm       Y = (X - mean) rstd gamma + beta;  with save: mean, rstd
  layer_norm_backward  dX, dgamma, dbeta
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
EPS = 1e-5
GELU_C = math.sqrt(2.0 / math.pi)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One decoded token through a square projection, in place on the
        # residual stream: the smallest call, all latency and weight reads.
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "M": 1, "N": 4096, "K": 4096,
         "act": "none", "bias": True, "residual": True, "save": False, "pad": 0},
        # The down projection of a large prefill batch with the residual added.
        {"name": "linear_down_8192", "op": "linear", "dtype": "bf16", "M": 8192, "N": 4096,
         "K": 14336, "act": "none", "bias": True, "residual": True, "save": False, "pad": 0},
        # A training step's ragged token count through a GELU layer that keeps
        # its pre-activations, on rows with stride padding.
        {"name": "linear_gelu_ragged", "op": "linear", "dtype": "fp16", "M": 1111, "N": 8200,
         "K": 2056, "act": "gelu_tanh", "bias": True, "residual": False, "save": True, "pad": 8},
        # The same layer kind's backward pass at a training batch's size.
        {"name": "linear_backward_4096", "op": "linear_backward", "dtype": "bf16", "M": 4096,
         "N": 16384, "K": 4096, "act": "gelu_tanh", "bias": True, "pad": 0},
        # Odd feature counts, whose rows start at odd 2-byte addresses.
        {"name": "linear_backward_odd", "op": "linear_backward", "dtype": "fp16", "M": 777,
         "N": 1001, "K": 1365, "act": "relu", "bias": True, "pad": 0},
        # Decoding: four sequences' new tokens through the gated unit.
        {"name": "gated_tokens", "op": "gated", "dtype": "bf16", "M": 4, "N": 14336, "K": 4096,
         "act": "silu", "save": False, "pad": 0},
        # A short ragged prompt.
        {"name": "gated_prompt", "op": "gated", "dtype": "fp16", "M": 333, "N": 5640, "K": 2048,
         "act": "gelu_tanh", "save": False, "pad": 0},
        # A training step's forward pass, which keeps both projections.
        {"name": "gated_train_8192", "op": "gated", "dtype": "bf16", "M": 8192, "N": 14336,
         "K": 4096, "act": "silu", "save": True, "pad": 0},
        # Its backward pass: the largest case.
        {"name": "gated_backward_8192", "op": "gated_backward", "dtype": "bf16", "M": 8192,
         "N": 14336, "K": 4096, "act": "silu", "pad": 0},
        # Decoding: a few tokens' norm.
        {"name": "norm_tokens", "op": "layer_norm", "dtype": "bf16", "M": 8, "N": 4096,
         "affine": True, "save": False, "pad": 0},
        # A training batch's norm, backward with the weight's gradient.
        {"name": "norm_backward_8192", "op": "layer_norm_backward", "dtype": "bf16", "M": 16384,
         "N": 4096, "affine": True, "pad": 0},
        # FP32 activations with an odd row length.
        {"name": "norm_backward_odd", "op": "layer_norm_backward", "dtype": "f32", "M": 4099,
         "N": 1001, "affine": True, "pad": 0},
    ]


# The largest listed case's operations and the largest norm's elements.
MOST_FLOPS = 8.0 * 8192 * 14336 * 4096
MOST_NORM = 16384 * 4096


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _features(rng, lo, hi):
    """A feature count: mostly a multiple of 64 or 8, sometimes any number."""
    unit = rng.choice([64, 64, 8, 8, 1])
    n = _spread(rng, lo, hi)
    n = max(unit, n // unit * unit)
    return n + unit if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "gated", "gated", "gated_backward",
                     "layer_norm", "layer_norm_backward"])
    if op.startswith("layer_norm"):
        case = {"op": op, "dtype": rng.choice(["bf16", "fp16", "f32"])}
        while True:
            case["M"], case["N"] = _spread(rng, 1, 16384), _features(rng, 64, 16384)
            if case["M"] * case["N"] <= MOST_NORM:
                break
        case["affine"] = rng.random() < 0.8
        if op == "layer_norm":
            case["save"] = rng.random() < 0.5
        case["pad"] = rng.choice([0, 0, 8, 3])
        return case
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    while True:
        case["M"] = _spread(rng, 1, 8192)
        case["N"], case["K"] = _features(rng, 256, 16384), _features(rng, 256, 14336)
        if work(dict(case, act="silu", bias=True, residual=True, save=True))["flops"] <= MOST_FLOPS:
            break
    if op.startswith("linear"):
        case["act"] = rng.choice(["none", "relu", "silu", "gelu_tanh"])
        case["bias"] = rng.random() < 0.7
    else:
        case["act"] = rng.choice(["silu", "silu", "gelu_tanh", "relu", "none"])
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    if op in ("linear", "gated"):
        case["save"] = rng.random() < 0.3
    case["pad"] = rng.choice([0, 0, 0, 8, 64, 5])
    return case


def work(case):
    op, m, n = case["op"], case["M"], case["N"]
    if op.startswith("layer_norm"):
        e = 4 if case["dtype"] == "f32" else 2
        a = 1 if case["affine"] else 0
        if op == "layer_norm":
            return {"bytes": 2 * m * n * e + 8 * n * a + (8 * m if case["save"] else 0),
                    "flops": 8 * m * n}
        return {"bytes": 3 * m * n * e + 12 * n * a + 8 * m, "flops": 14 * m * n}
    k = case["K"]
    if op == "linear":
        outs = m * n * (1 + int(case["residual"]) + int(case["save"]))
        return {"bytes": 2 * (m * k + n * k + outs) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "linear_backward":
        z = 0 if case["act"] == "none" else m * n
        return {"bytes": 2 * (m * n + z + 2 * m * k + 2 * n * k) + (4 * n if case["bias"] else 0),
                "flops": 4 * m * n * k}
    if op == "gated":
        outs = m * n * (3 if case["save"] else 1)
        return {"bytes": 2 * (m * k + 2 * n * k + outs), "flops": 4 * m * n * k}
    return {"bytes": 2 * (3 * m * n + 2 * m * k + 4 * n * k), "flops": 8 * m * n * k}


# ------------------------------------------------------------------ inputs


def _matrix(g, rows, cols, dtype, pad, scale=1.0, shift=0.0):
    """rows x cols values of a wider buffer whose padding holds NaN."""
    buf = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")
    if pad:
        buf[:, cols:] = float("nan")
    buf[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda").mul_(scale).add_(shift)
    return buf[:, :cols]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, m, n, pad = TYPES[case["dtype"]], case["M"], case["N"], case["pad"]
    op = case["op"]
    if op.startswith("layer_norm"):
        s = {"X": _matrix(g, m, n, t, pad, 1.5, 0.25)}
        if case["affine"]:
            s["gamma"] = 1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")
            s["beta"] = 0.2 * torch.randn(n, generator=g, device="cuda")
        if op == "layer_norm_backward":
            s["dY"] = _matrix(g, m, n, t, pad, 0.5)
            x = s["X"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        return s
    k = case["K"]
    w = 1.0 / math.sqrt(k)
    s = {"X": _matrix(g, m, k, t, pad)}
    if op.startswith("linear"):
        s["W"] = _matrix(g, n, k, t, pad, w)
        if case["bias"]:
            s["bias"] = 0.1 * torch.randn(n, generator=g, device="cuda")
        if op == "linear":
            if case["residual"]:
                s["R"] = _matrix(g, m, n, t, pad)
        else:
            s["dY"] = _matrix(g, m, n, t, pad, 0.5)
            if case["act"] != "none":
                s["Z"] = _matrix(g, m, n, t, pad)
                s["Z"].copy_(s["X"] @ s["W"].t())
        return s
    s["Wg"] = _matrix(g, n, k, t, pad, w)
    s["Wu"] = _matrix(g, n, k, t, pad, w)
    if op == "gated_backward":
        s["dH"] = _matrix(g, m, n, t, pad, 0.5)
        s["G"] = _matrix(g, m, n, t, pad)
        s["U"] = _matrix(g, m, n, t, pad)
        s["G"].copy_(s["X"] @ s["Wg"].t())
        s["U"].copy_(s["X"] @ s["Wu"].t())
    return s


def prepare(case, seed):
    """The inputs and the buffers that the outputs go to."""
    s = {"case": case, "in": _inputs(case, seed)}
    m, n, t, op = case["M"], case["N"], TYPES[case["dtype"]], case["op"]

    def out(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    f32 = torch.float32
    if op == "linear":
        s["out"] = {"Y": out(m, n)}
        if case["save"]:
            s["out"]["Z"] = out(m, n)
    elif op == "linear_backward":
        s["out"] = {"dX": out(m, case["K"]), "dW": out(n, case["K"])}
        if case["bias"]:
            s["out"]["db"] = out(n, dtype=f32)
    elif op == "gated":
        s["out"] = {"H": out(m, n)}
        if case["save"]:
            s["out"] |= {"G": out(m, n), "U": out(m, n)}
    elif op == "gated_backward":
        s["out"] = {"dX": out(m, case["K"]), "dWg": out(n, case["K"]), "dWu": out(n, case["K"])}
    elif op == "layer_norm":
        s["out"] = {"Y": out(m, n)}
        if case["save"]:
            s["out"] |= {"mean": out(m, dtype=f32), "rstd": out(m, dtype=f32)}
    else:
        s["out"] = {"dX": out(m, n)}
        if case["affine"]:
            s["out"] |= {"dgamma": out(n, dtype=f32), "dbeta": out(n, dtype=f32)}
    return s


# ------------------------------------------------------------------ the plain form


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(name, x):
    if name == "none":
        return x
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x * _sigmoid(x)
    return 0.5 * x * (1.0 + torch.tanh(GELU_C * (x + 0.044715 * x * x * x)))


def _act_grad(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        s = _sigmoid(x)
        return s * (1.0 + x * (1.0 - s))
    t = torch.tanh(GELU_C * (x + 0.044715 * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * GELU_C * (1.0 + 3 * 0.044715 * x * x)


def _plain(case, i):
    op, t = case["op"], TYPES[case["dtype"]]
    x = i["X"].float()
    if op == "linear":
        z = x @ i["W"].float().t()
        if case["bias"]:
            z = z + i["bias"]
        y = _act(case["act"], z)
        if case["residual"]:
            y = y + i["R"].float()
        return {"Y": y.to(t), "Z": z.to(t)} if case["save"] else {"Y": y.to(t)}
    if op == "linear_backward":
        dz = i["dY"].float()
        if case["act"] != "none":
            dz = dz * _act_grad(case["act"], i["Z"].float())
        o = {"dX": (dz @ i["W"].float()).to(t), "dW": (dz.t() @ x).to(t)}
        if case["bias"]:
            o["db"] = dz.sum(0)
        return o
    if op == "gated":
        g, u = x @ i["Wg"].float().t(), x @ i["Wu"].float().t()
        h = _act(case["act"], g) * u
        return {"H": h.to(t), "G": g.to(t), "U": u.to(t)} if case["save"] else {"H": h.to(t)}
    if op == "gated_backward":
        dh, g, u = i["dH"].float(), i["G"].float(), i["U"].float()
        dg, du = dh * u * _act_grad(case["act"], g), dh * _act(case["act"], g)
        return {"dX": (dg @ i["Wg"].float() + du @ i["Wu"].float()).to(t),
                "dWg": (dg.t() @ x).to(t), "dWu": (du.t() @ x).to(t)}
    if op == "layer_norm":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd
        if case["affine"]:
            y = y * i["gamma"] + i["beta"]
        o = {"Y": y.to(t)}
        if case["save"]:
            o |= {"mean": mean[:, 0], "rstd": rstd[:, 0]}
        return o
    dy, rstd = i["dY"].float(), i["rstd"][:, None]
    xh = (x - i["mean"][:, None]) * rstd
    a = dy * i["gamma"] if case["affine"] else dy
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    o = {"dX": dx.to(t)}
    if case["affine"]:
        o |= {"dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    return o


# ------------------------------------------------------------------ the framework's calls


def _ld(x):
    return x.stride(0) if x is not None else 0


def _space(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def _framework(case, i, o):
    import dense_gemm_epilogue_gb300 as tg

    st = torch.cuda.current_stream()
    op, t, m, n = case["op"], case["dtype"], case["M"], case["N"]
    x = i["X"]
    if op == "layer_norm":
        y, mean, rstd = o["Y"], o.get("mean"), o.get("rstd")
        tg.check(tg.tg_layer_norm(m, n, x, _ld(x), i.get("gamma"), i.get("beta"), EPS, y, _ld(y),
                                  mean, rstd, t, st))
        return o
    if op == "layer_norm_backward":
        dy, dx = i["dY"], o["dX"]
        ws = _space(tg.tg_layer_norm_backward_workspace_bytes(m, n))
        tg.check(tg.tg_layer_norm_backward(m, n, dy, _ld(dy), x, _ld(x), i.get("gamma"), i["mean"],
                                           i["rstd"], dx, _ld(dx), o.get("dgamma"), o.get("dbeta"),
                                           t, ws, st))
        return o
    k, act = case["K"], case["act"]
    if op == "linear":
        w, r, y, z = i["W"], i.get("R"), o["Y"], o.get("Z")
        ws = _space(tg.tg_linear_workspace_bytes(m, n, k, x, _ld(x), w, _ld(w), t))
        tg.check(tg.tg_linear(m, n, k, x, _ld(x), w, _ld(w), i.get("bias"), act, r, _ld(r), y,
                              _ld(y), z, _ld(z), t, ws, st))
    elif op == "linear_backward":
        w, dy, z, dx, dw = i["W"], i["dY"], i.get("Z"), o["dX"], o["dW"]
        ws = _space(tg.tg_linear_backward_workspace_bytes(m, n, k, dy, _ld(dy), x, _ld(x), w,
                                                          _ld(w), act, t))
        tg.check(tg.tg_linear_backward(m, n, k, dy, _ld(dy), x, _ld(x), w, _ld(w), z, _ld(z), act,
                                       dx, _ld(dx), dw, _ld(dw), t, o.get("db"), t, ws, st))
    elif op == "gated":
        wg, wu, h, g, u = i["Wg"], i["Wu"], o["H"], o.get("G"), o.get("U")
        ws = _space(tg.tg_gated_workspace_bytes(m, n, k, x, _ld(x), wg, _ld(wg), wu, _ld(wu), t))
        tg.check(tg.tg_gated(m, n, k, x, _ld(x), wg, _ld(wg), wu, _ld(wu), act, h, _ld(h), g,
                             _ld(g), u, _ld(u), t, ws, st))
    else:
        wg, wu, dh, g, u = i["Wg"], i["Wu"], i["dH"], i["G"], i["U"]
        dx, dwg, dwu = o["dX"], o["dWg"], o["dWu"]
        ws = _space(tg.tg_gated_backward_workspace_bytes(m, n, k, x, _ld(x), wg, _ld(wg), wu,
                                                         _ld(wu), t))
        tg.check(tg.tg_gated_backward(m, n, k, dh, _ld(dh), x, _ld(x), wg, _ld(wg), wu, _ld(wu), g,
                                      _ld(g), u, _ld(u), act, dx, _ld(dx), dwg, _ld(dwg), dwu,
                                      _ld(dwu), t, t, ws, st))
    return o


def run(state):
    if own:
        return _framework(state["case"], state["in"], state["out"])
    return _plain(state["case"], state["in"])


# ------------------------------------------------------------------ the definitions in 64 bits


def _e_act(name, x):
    """(act(x), act'(x)) in FP64; the tanh form of GELU is x times the
    logistic function of twice its argument."""
    if name == "none":
        return x, torch.full_like(x, 1.0)
    if name == "relu":
        on = torch.gt(x, 0).double()
        return x.clamp(min=0), on
    if name == "silu":
        s = x.sigmoid()
        return x * s, s + x * s * (1 - s)
    v = 2 * GELU_C * (x + 0.044715 * x.pow(3))
    s = v.sigmoid()
    return x * s, s + x * s * (1 - s) * (2 * GELU_C * (1 + 0.134145 * x.pow(2)))


def exact(case, seed):
    i = {name: v.double() for name, v in _inputs(case, seed).items()}
    op, x = case["op"], i["X"]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", x, i["W"]) + i.get("bias", 0.0)
        o = {"Y": _e_act(case["act"], z)[0] + i.get("R", 0.0)}
        if case["save"]:
            o["Z"] = z
        return o
    if op == "linear_backward":
        dz = i["dY"] * _e_act(case["act"], i["Z"])[1] if "Z" in i else i["dY"]
        o = {"dX": torch.einsum("mn,nk->mk", dz, i["W"]), "dW": torch.einsum("mn,mk->nk", dz, x)}
        if case["bias"]:
            o["db"] = torch.einsum("mn->n", dz)
        return o
    if op == "gated":
        g = torch.einsum("mk,nk->mn", x, i["Wg"])
        u = torch.einsum("mk,nk->mn", x, i["Wu"])
        o = {"H": _e_act(case["act"], g)[0] * u}
        if case["save"]:
            o |= {"G": g, "U": u}
        return o
    if op == "gated_backward":
        a, da = _e_act(case["act"], i["G"])
        dg, du = i["dH"] * i["U"] * da, i["dH"] * a
        return {"dX": torch.einsum("mn,nk->mk", dg, i["Wg"]) + torch.einsum("mn,nk->mk", du, i["Wu"]),
                "dWg": torch.einsum("mn,mk->nk", dg, x), "dWu": torch.einsum("mn,mk->nk", du, x)}
    n = case["N"]
    if op == "layer_norm":
        mean = torch.einsum("mn->m", x) / n
        var = torch.einsum("mn,mn->m", x, x) / n - mean.square()
        rstd = (var + EPS).pow(-0.5)
        y = torch.einsum("mn,m->mn", x - mean[:, None], rstd)
        if case["affine"]:
            y = y * i["gamma"] + i["beta"]
        return {"Y": y, "mean": mean, "rstd": rstd} if case["save"] else {"Y": y}
    xh = torch.einsum("mn,m->mn", x - i["mean"][:, None], i["rstd"])
    a = i["dY"] * i.get("gamma", torch.ones(n, dtype=torch.float64, device="cuda"))
    p, q = torch.einsum("mn->m", a) / n, torch.einsum("mn,mn->m", a, xh) / n
    o = {"dX": torch.einsum("mn,m->mn", a - p[:, None] - xh * q[:, None], i["rstd"])}
    if case["affine"]:
        o |= {"dgamma": torch.einsum("mn,mn->n", i["dY"], xh), "dbeta": torch.einsum("mn->n", i["dY"])}
    return o
