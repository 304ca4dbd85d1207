"""The dense operators beside the routed experts: cases, inputs, and the operators' plain forms.

Two operators, each forward and backward (row-major matrices, one row per token; W is [n_out][n_in]):

  linear   z = x W^T + b,  y = act(z) + r
           dz = dy * act'(z),  dx = dz W,  dW = dz^T x,  db = sum_t dz
  gated    g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) * u
           dg = dh * u * act'(g),  du = dh * act(g),
           dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dbg = sum_t dg,  dbu = sum_t du

The backward passes take the pre-activations (z; g and u) that a forward pass has saved in the
operands' type.  ``own`` chooses between the plain forms below and the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid")

MAX_FLOPS = 1.1e12   # the largest listed case (the backward pass of the wide gated block)
MAX_VALUES = 6.0e8   # values read and written by the largest listed case


def _case(name, op, tokens, n_in, n_out, dtype="bf16", act="none", bias=False, residual="none", y="same",
          save=False, x_pad=0):
    """residual: none, same (the operands' type) or f32 (with y = f32).  x_pad: x is a slice of rows
    that are this many elements wider."""
    return {"name": name, "op": op, "tokens": tokens, "n_in": n_in, "n_out": n_out, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "y": y, "save": save, "x_pad": x_pad}


def listed():
    return [
        # one token through an expert-sized gated block and back down onto the routed layer's fp32 output:
        # the two calls of a dense shared expert in a decode step, where latency counts
        _case("gated_1tok", "gated_forward", 1, 2048, 768, act="silu"),
        _case("linear_1tok_onto_f32", "linear_forward", 1, 768, 2048, residual="f32", y="f32"),
        # a decode batch through the wide dense block of a model's first layers
        _case("gated_8tok_wide", "gated_forward", 8, 2048, 8192, act="silu"),
        _case("linear_16tok_wide", "linear_forward", 16, 8192, 2048, bias=True, residual="same"),
        # the output head of a small decode batch: an odd vocabulary, fp32 logits
        _case("linear_head_5tok", "linear_forward", 5, 2048, 100003, y="f32"),
        # a short prompt, odd widths, another activation, fp16
        _case("gated_333tok_odd", "gated_forward", 333, 1000, 1357, dtype="fp16", act="gelu_tanh", bias=True),
        # a prompt chunk through the wide block, and a training forward that saves what its backward needs
        _case("gated_4096tok_wide", "gated_forward", 4096, 2048, 8192, act="silu", save=True),
        _case("linear_4096tok_wide", "linear_forward", 4096, 8192, 2048, residual="same"),
        _case("linear_2500tok_gelu", "linear_forward", 2500, 4096, 4096, act="gelu", bias=True, save=True),
        # training: the backward passes, wide and odd
        _case("gated_bwd_8192tok_wide", "gated_backward", 8192, 2048, 8192, act="silu"),
        _case("linear_bwd_8192tok_wide", "linear_backward", 8192, 8192, 2048, bias=True),
        _case("linear_bwd_333tok_odd", "linear_backward", 333, 1000, 1357, dtype="fp16", act="gelu", bias=True),
    ]


def _width(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.5:
        v = max(lo, v // 128 * 128)
    elif kind < 0.75:
        v = max(lo, v // 8 * 8)
    return v


def draw(rng):
    """The listed ranges: 1 to 8192 tokens, widths 128 to 8192 (an output head up to 131072), every type,
    activation and epilogue; half the widths whole multiples of 128, a quarter any number at all."""
    while True:
        op = rng.choice(("gated_forward", "gated_backward", "linear_forward", "linear_backward"))
        tokens = int(round(math.exp(rng.uniform(0.0, math.log(8192.0)))))
        if op.endswith("backward"):
            tokens = max(tokens, int(round(math.exp(rng.uniform(0.0, math.log(8192.0))))))
        n_in = _width(rng, 128, 8192)
        head = op == "linear_forward" and rng.random() < 0.2
        n_out = _width(rng, 8192, 131072) if head else _width(rng, 128, 8192)
        dtype = "bf16" if rng.random() < 0.7 else "fp16"
        act = rng.choice(ACTS[1:]) if op.startswith("gated") or rng.random() < 0.5 else "none"
        y = residual = "same"
        if op == "linear_forward":
            y = "f32" if head or rng.random() < 0.3 else "same"
        residual = y if op == "linear_forward" and rng.random() < 0.4 else "none"
        case = _case("", op, tokens, n_in, n_out, dtype, act, rng.random() < 0.5, residual, y,
                     op.endswith("forward") and (op.startswith("gated") or act != "none") and rng.random() < 0.4,
                     rng.choice((0, 0, 8, 3)))
        del case["name"]
        w = work(case)
        if w["flops"] <= MAX_FLOPS and _values(case) <= MAX_VALUES:
            return case


def _mats(case):
    return 2 if case["op"].startswith("gated") else 1


def _values(case):
    t, k, n, m = case["tokens"], case["n_in"], case["n_out"], _mats(case)
    return (2 * t * k + 2 * m * n * k + (2 * m + 1) * t * n) if case["op"].endswith("backward") else \
        (t * k + m * n * k + 3 * t * n)


def work(case):
    """Bytes: each input read once, each output written once.  Flops: the matrix products."""
    t, k, n, m = case["tokens"], case["n_in"], case["n_out"], _mats(case)
    wide = 4 if case["y"] == "f32" else 2
    if case["op"].endswith("forward"):
        elems = t * k + m * n * k + (m * n if case["bias"] else 0) + (m * t * n if case["save"] else 0)
        out = t * n * wide + (t * n * wide if case["residual"] != "none" else 0)
        return {"bytes": 2 * elems + out, "flops": 2 * m * t * n * k}
    pre = m * t * n if (m == 2 or case["act"] != "none") else 0
    elems = 2 * t * k + 2 * m * n * k + pre + t * n + (m * n if case["bias"] else 0)
    return {"bytes": 2 * elems, "flops": 4 * m * t * n * k}


# ---- the activations and their derivatives, elementary operations ---------------------------------

def _act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * (1.0 / math.sqrt(2.0))))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return 1.0 / (1.0 + torch.exp(-z))


def _dact(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * (1.0 / math.sqrt(2.0)))) + \
            z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 - s)


# ---- inputs ---------------------------------------------------------------------------------------

def prepare(case, seed):
    """Normalised activations, weights of variance 1 / n_in, gradients a tenth of the activations; the
    saved pre-activations are the forward pass's own, rounded to the operands' type."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2654435761 % (2 ** 31) + 17)
    dt = DTYPES[case["dtype"]]
    t, k, n, m = case["tokens"], case["n_in"], case["n_out"], _mats(case)

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": case, "x": normal(t, k + case["x_pad"])[:, :k]}
    s["w"] = [normal(n, k, scale=1.0 / math.sqrt(k)) for _ in range(m)]
    s["b"] = [normal(n, scale=0.1) if case["bias"] else None for _ in range(m)]
    s["r"] = None
    if case["op"].endswith("forward"):
        if case["residual"] != "none":
            s["r"] = normal(t, n, dtype=torch.float32 if case["y"] == "f32" else dt)
    else:
        s["dy"] = normal(t, n, scale=0.1)
        s["pre"] = [None]
        if m == 2 or case["act"] != "none":
            s["pre"] = [_linear32(s["x"], s["w"][i], s["b"][i]).to(dt) for i in range(m)]
    if own:
        _prepare_own(s)
    return s


def _linear32(x, w, b):
    z = x.float() @ w.float().t()
    return z if b is None else z + b.float()


# ---- the plain forms ------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    case, act = state["case"], state["case"]["act"]
    x, w, b = state["x"], state["w"], state["b"]
    dt = x.dtype
    if case["op"] == "linear_forward":
        z = _linear32(x, w[0], b[0])
        y = _act(act, z)
        if state["r"] is not None:
            y = y + state["r"].float()
        out = {"y": y if case["y"] == "f32" else y.to(dt)}
        if case["save"]:
            out["pre"] = z.to(dt)
        return out
    if case["op"] == "gated_forward":
        g, u = _linear32(x, w[0], b[0]), _linear32(x, w[1], b[1])
        out = {"h": (_act(act, g) * u).to(dt)}
        if case["save"]:
            out["gate"], out["up"] = g.to(dt), u.to(dt)
        return out
    dy = state["dy"].float()
    if case["op"] == "linear_backward":
        dz = [dy if act == "none" else dy * _dact(act, state["pre"][0].float())]
    else:
        g, u = state["pre"][0].float(), state["pre"][1].float()
        dz = [dy * u * _dact(act, g), dy * _act(act, g)]
    dx = dz[0] @ w[0].float()
    for i in range(1, len(dz)):
        dx = dx + dz[i] @ w[i].float()
    xf = x.float()
    out = {"dx": dx.to(dt), "dw": [d.t() @ xf for d in dz]}
    out["dw"] = [d.to(dt) for d in out["dw"]]
    if case["bias"]:
        out["db"] = [d.sum(dim=0).to(dt) for d in dz]
    return out


# ---- the library's entry points -------------------------------------------------------------------

def _prepare_own(s):
    from mixture_experts_route_amd import native as N

    case, x = s["case"], s["x"]
    dt, dev = x.dtype, x.device
    t, k, n = case["tokens"], case["n_in"], case["n_out"]
    backward = case["op"].endswith("backward")
    s["act"] = getattr(N, "MOE_ACT_" + case["act"].upper())
    s["d"] = N.dense_dims(k, n, N.dtype_code(x), s["act"])
    nbytes = N.moe_dense_workspace_bytes(s["d"], t, backward)
    s["ws"] = torch.empty((nbytes + 3) // 4, dtype=torch.int32, device=dev)
    N.moe_workspace_init(s["ws"])
    s["out"] = {}
    if case["op"] == "linear_forward":
        s["out"]["y"] = torch.empty((t, n), dtype=torch.float32 if case["y"] == "f32" else dt, device=dev)
        if case["save"]:
            s["out"]["pre"] = torch.empty((t, n), dtype=dt, device=dev)
    elif case["op"] == "gated_forward":
        s["out"]["h"] = torch.empty((t, n), dtype=dt, device=dev)
        if case["save"]:
            s["out"]["gate"] = torch.empty((t, n), dtype=dt, device=dev)
            s["out"]["up"] = torch.empty((t, n), dtype=dt, device=dev)
    else:
        s["out"]["dx"] = torch.empty((t, k), dtype=dt, device=dev)
        s["out"]["dw"] = [torch.empty((n, k), dtype=dt, device=dev) for _ in s["w"]]
        if case["bias"]:
            s["out"]["db"] = [torch.empty((n,), dtype=dt, device=dev) for _ in s["w"]]


def _run_own(s):
    from mixture_experts_route_amd import native as N

    case, out, d, ws = s["case"], s["out"], s["d"], s["ws"]
    t, x, w, b = case["tokens"], s["x"], s["w"], s["b"]
    if case["op"] == "linear_forward":
        N.moe_linear_forward(d, x, t, w[0], out["y"], ws, bias=b[0], residual=s["r"], pre=out.get("pre"))
    elif case["op"] == "gated_forward":
        N.moe_gated_forward(d, x, t, w[0], w[1], out["h"], ws, gate_bias=b[0], up_bias=b[1], gate=out.get("gate"),
                            up=out.get("up"))
    elif case["op"] == "linear_backward":
        N.moe_linear_backward(d, x, t, w[0], s["dy"], ws, pre=s["pre"][0], dx=out["dx"], dw=out["dw"][0],
                              dbias=out["db"][0] if case["bias"] else None)
    else:
        db = out["db"] if case["bias"] else (None, None)
        N.moe_gated_backward(d, x, t, w[0], w[1], s["pre"][0], s["pre"][1], s["dy"], ws, dx=out["dx"],
                             dw_gate=out["dw"][0], dw_up=out["dw"][1], dgate_bias=db[0], dup_bias=db[1])
    return out


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _exact_act(name, z):
    """(value, derivative) in float64, from the definitions."""
    one = torch.ones((), dtype=torch.float64, device=z.device)
    if name == "none":
        return z, one.expand_as(z)
    if name == "relu":
        return z.clamp(min=0.0), torch.heaviside(z, 0.0 * one)
    if name in ("silu", "sigmoid"):
        p = torch.special.expit(z)
        if name == "sigmoid":
            return p, p * torch.special.expit(-z)
        return z * p, p + z * p * torch.special.expit(-z)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2.0) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(8.0 / math.pi)  # (1 + tanh(v)) / 2 = expit(2 v)
    p = torch.special.expit(a * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1.0 - p) * a * (1.0 + 0.134145 * z.square())


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    w = [v.double() for v in s["w"]]
    b = [None if v is None else v.double() for v in s["b"]]
    if case["op"].endswith("forward"):
        z = [torch.matmul(x, v.T) if c is None else torch.addmm(c, x, v.T) for v, c in zip(w, b)]
        a = _exact_act(case["act"], z[0])[0]
        if case["op"] == "gated_forward":
            out = {"h": a.mul(z[1])}
            if case["save"]:
                out.update(gate=z[0], up=z[1])
            return out
        out = {"y": a if s["r"] is None else a.add(s["r"].double())}
        if case["save"]:
            out["pre"] = z[0]
        return out
    dy = s["dy"].double()
    if case["op"] == "gated_backward":
        a, da = _exact_act(case["act"], s["pre"][0].double())
        dz = [da.mul_(s["pre"][1].double()).mul_(dy), a.mul_(dy)]
    elif case["act"] == "none":
        dz = [dy]
    else:
        dz = [_exact_act(case["act"], s["pre"][0].double())[1].mul(dy)]
    dx = torch.matmul(dz[0], w[0])
    for i in range(1, len(dz)):
        dx.addmm_(dz[i], w[i])
    out = {"dx": dx, "dw": [torch.matmul(d.T, x) for d in dz]}
    if case["bias"]:
        out["db"] = [d.sum(0) for d in dz]
    return out
