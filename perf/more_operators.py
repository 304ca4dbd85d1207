"""Training the routed layer with 16-bit experts, and the loss over the output head: cases, inputs, and the
operators' plain forms.

Pairs p = t k + j are a token's choices; perm[r] is the pair in row r of the rows sorted by expert (-1: a padding
row), inv[p] the row of pair p (-1: dropped); rows offsets[e] .. offsets[e+1]-1 belong to expert e.

  dispatch   xs[r] = x[perm[r] / k] (0 in padding rows), inv          dx[t] = sum_j dxs[inv[t,j]] + r[t]
  combine    y[t] = sum_j w[t,j] ys[inv[t,j]] + r[t]
             dys[r] = w[perm[r]] dy[perm[r] / k],  dw[t,j] = <dy[t], ys[inv[t,j]]>
  experts    linear y_r = W_e x_r; gated g_r = Wg_e x_r, u_r = Wu_e x_r, h_r = act(g_r) * u_r
             linear dx_r = W_e^T dy_r, dW_e = sum_r dy_r x_r^T
             gated dg = dh * u * act'(g), du = dh * act(g), dx_r = Wg_e^T dg_r + Wu_e^T du_r, dWg_e, dWu_e
  loss       z = x W^T, loss_t = log sum_v exp(z_tv) - z_t,target, lse_t = loss_t + z_t,target (0 where ignored)
             dz_tv = dloss_t (exp(z_tv - lse_t) - [v = target]), dx = dz W, dW = dz^T x

The backward passes take what a forward pass has saved (inv; g and u; loss and lse).  ``own`` chooses between the
plain forms below and the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
IGNORE = -100

MAX_FLOPS = 1.01e13   # the largest listed case (the loss's backward pass)
MAX_BYTES = 6.9e9     # the largest listed case (the experts' gated backward pass)
MAX_ROW_BYTES = 1.6e9  # the largest listed case that only moves rows


def _rows(name, op, tokens, top_k, experts, width, dtype="bf16", y="same", residual=False, pad=1, drop=False, x_pad=0):
    """pad: groups padded to a multiple of so many rows.  drop: an expert takes at most twice the mean.  x_pad: the
    token rows are slices of rows that are this many elements wider."""
    return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "width": width, "dtype": dtype,
            "y": y, "residual": residual, "pad": pad, "drop": drop, "x_pad": x_pad}


def _experts(name, op, tokens, top_k, experts, n_in, n_out, dtype="bf16", act="none", save=False):
    return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "n_in": n_in, "n_out": n_out,
            "dtype": dtype, "act": act, "save": save}


def _loss(name, op, tokens, n_in, vocab, dtype="bf16"):
    return {"name": name, "op": op, "tokens": tokens, "n_in": n_in, "vocab": vocab, "dtype": dtype}


def listed():
    return [
        # a small decode batch's rows laid out by expert: the smallest call, where latency counts
        _rows("dispatch_8tok", "dispatch_forward", 8, 10, 512, 2048),
        # the gradient of a long batch's rows back to its tokens, onto the shared expert's gradient
        _rows("dispatch_bwd_32768tok", "dispatch_backward", 32768, 10, 512, 2048, residual=True),
        # a prompt chunk's expert outputs weighted and added onto the layer's fp32 stream
        _rows("combine_4096tok_f32", "combine_forward", 4096, 10, 512, 2048, y="f32", residual=True),
        # the gradients of the expert outputs and of the router weights; odd width, padded groups, dropped pairs
        _rows("combine_bwd_8191tok_odd", "combine_backward", 8191, 4, 60, 1357, dtype="fp16", pad=16, drop=True, x_pad=3),
        # one token through its ten unquantized experts: bound by ten experts' weights
        _experts("experts_gated_1tok", "experts_gated_forward", 1, 10, 512, 2048, 768, act="silu"),
        # a training batch through the experts, forward (saving what the backward needs) and down
        _experts("experts_gated_4096tok", "experts_gated_forward", 4096, 10, 512, 2048, 768, act="silu", save=True),
        _experts("experts_linear_4096tok", "experts_linear_forward", 4096, 10, 512, 768, 2048),
        # the gradients of that batch
        _experts("experts_gated_bwd_4096tok", "experts_gated_backward", 4096, 10, 512, 2048, 768, act="silu"),
        # few experts, odd widths, fp16
        _experts("experts_linear_bwd_333tok_odd", "experts_linear_backward", 333, 2, 24, 1000, 1357, dtype="fp16"),
        # scoring a few tokens against an odd vocabulary: bound by the head's weights
        _loss("loss_5tok", "loss_forward", 5, 2048, 100003),
        # a short odd batch, fp16
        _loss("loss_333tok_odd", "loss_forward", 333, 1000, 32771, dtype="fp16"),
        # a training batch's gradients
        _loss("loss_bwd_8192tok", "loss_backward", 8192, 2048, 100003),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    v = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.5:
        v = max(lo, v // 128 * 128)
    elif kind < 0.75:
        v = max(lo, v // 8 * 8)
    return v


def draw(rng):
    """The listed ranges: 1 to 32768 tokens (experts and loss: 8192), 1 to 10 choices of 4 to 512 experts, widths 64 to
    8192 (half of them whole multiples of 128, a quarter any number at all), vocabularies up to 131072."""
    while True:
        op = rng.choice(("dispatch_forward", "dispatch_backward", "combine_forward", "combine_backward",
                         "experts_gated_forward", "experts_linear_forward", "experts_gated_backward",
                         "experts_linear_backward", "loss_forward", "loss_backward"))
        dtype = "bf16" if rng.random() < 0.7 else "fp16"
        experts = _log(rng, 4, 512)
        top_k = rng.randint(1, min(10, experts))
        if op.startswith("loss"):
            case = _loss("", op, _log(rng, 1, 8192), _width(rng, 64, 4096), _width(rng, 64, 131072), dtype)
        elif op.startswith("experts"):
            act = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu", "sigmoid")) if "gated" in op else "none"
            case = _experts("", op, _log(rng, 1, 8192), top_k, experts, _width(rng, 64, 4096), _width(rng, 64, 4096), dtype,
                            act, op == "experts_gated_forward" and rng.random() < 0.5)
        else:
            y = "f32" if op.startswith("combine") and rng.random() < 0.5 else "same"
            residual = op in ("dispatch_backward", "combine_forward") and rng.random() < 0.5
            case = _rows("", op, _log(rng, 1, 32768), top_k, experts, _width(rng, 64, 8192), dtype, y, residual,
                         rng.choice((1, 1, 16)), rng.random() < 0.3, rng.choice((0, 0, 8, 3)))
        del case["name"]
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= (MAX_ROW_BYTES if "width" in case else MAX_BYTES):
            return case


def _touched(case):
    """Experts that have rows, about: each choice of every token a uniform one (in use they are skewed, so fewer)."""
    return case["experts"] * (1.0 - (1.0 - case["top_k"] / case["experts"]) ** case["tokens"])


def work(case):
    """Bytes: each input read once, each output written once.  Flops: the matrix products."""
    op, t = case["op"], case["tokens"]
    if op.startswith("loss"):
        k, v = case["n_in"], case["vocab"]
        if op == "loss_forward":
            return {"bytes": 2 * (t * k + v * k) + 12 * t, "flops": 2 * t * k * v}
        return {"bytes": 4 * (t * k + v * k) + 16 * t, "flops": 6 * t * k * v}
    pairs = t * case["top_k"]
    if op.startswith("experts"):
        k, n, m = case["n_in"], case["n_out"], 2 if "gated" in op else 1
        weights = m * int(_touched(case) * k * n)
        if op.endswith("forward"):
            elems = pairs * k + weights + pairs * n * (1 + (m if case["save"] else 0))
            return {"bytes": 2 * elems, "flops": 2 * m * pairs * k * n}
        elems = 2 * pairs * k + weights + m * case["experts"] * k * n + pairs * n * (1 + (2 if m == 2 else 0))
        return {"bytes": 2 * elems, "flops": 4 * m * pairs * k * n}
    h, wide = case["width"], 4 if case["y"] == "f32" else 2
    if op == "dispatch_forward":
        return {"bytes": 2 * h * (t + pairs) + 8 * pairs, "flops": 0}
    token = t * h * wide * (2 if case["residual"] else 1)
    if op == "dispatch_backward":
        return {"bytes": 2 * h * pairs + token + 4 * pairs, "flops": h * pairs}
    if op == "combine_forward":
        return {"bytes": 2 * h * pairs + token + 8 * pairs, "flops": 2 * h * pairs}
    return {"bytes": 4 * h * pairs + token + 16 * pairs, "flops": 3 * h * pairs}


# ---- inputs ---------------------------------------------------------------------------------------

def _route(case, gen, dev):
    """Distinct choices with a Zipf-like popularity, their softmax weights, and the sorted layout.  The number of rows is
    what a program allocates before it knows the counts: padding rows follow the last group."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    rank = torch.randperm(e, generator=gen, device=dev)
    logits = 0.9 * torch.randn(t, e, generator=gen, device=dev) - 0.46 * torch.log1p(rank.float())
    top, ids = logits.topk(k, dim=1)
    w = torch.softmax(top, dim=1)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=e)
    rank_in = torch.arange(t * k, device=dev) - (counts.cumsum(0) - counts)[flat[order]]
    pad, cap = case.get("pad", 1), max(1, 2 * t * k // e) if case.get("drop") else t * k
    kept = counts.clamp(max=cap)
    sizes = (kept + pad - 1) // pad * pad
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=dev)
    offsets[1:] = sizes.cumsum(0)
    n_rows = t * k + e * (pad - 1)
    keep = rank_in < cap
    perm = torch.full((n_rows,), -1, dtype=torch.int32, device=dev)
    perm[(offsets[:-1][flat[order]] + rank_in)[keep]] = order[keep].to(torch.int32)
    return perm, offsets.to(torch.int32), w, n_rows


def _invert(perm, pairs):
    """inv of a perm without repeated pairs; the padding rows write one element past the end, which is cut off."""
    inv = torch.full((pairs + 1,), -1, dtype=torch.int32, device=perm.device)
    at = torch.where(perm >= 0, perm, torch.full_like(perm, pairs)).long()
    inv[at] = torch.arange(perm.numel(), dtype=torch.int32, device=perm.device)
    return inv[:pairs]


def prepare(case, seed):
    """Normalised activations, weights of variance 1 / n_in, gradients a tenth of the activations; what a forward pass
    saves is that pass's own, rounded to its type."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2654435761 % (2 ** 31) + 29)
    dt, op, t = DTYPES[case["dtype"]], case["op"], case["tokens"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": case}
    if op.startswith("loss"):
        k, v = case["n_in"], case["vocab"]
        s["w"] = normal(v, k, scale=1.0 / math.sqrt(k))
        s["targets"] = torch.randint(0, v, (t,), generator=gen, device=dev, dtype=torch.int32)
        # a trained model's spread: each token's activation leans towards its target's row, some far enough to be sure
        lean = 6.0 * torch.rand(t, 1, generator=gen, device=dev) ** 2 * math.log(v) / 2.0
        s["x"] = (2.0 * normal(t, k, dtype=torch.float32) + lean * s["w"][s["targets"].long()].float()).to(dt)
        skip = torch.rand(t, generator=gen, device=dev) < 0.06  # a prompt's tokens and padding
        s["targets"][skip] = IGNORE
        if op == "loss_backward":
            s["loss"], s["lse"] = _loss32(s["x"], s["w"], s["targets"])
            # the mean over the tokens; fp16 training scales it
            s["dloss"] = torch.full((t,), (65536.0 if dt == torch.float16 else 1.0) / t, device=dev)
    elif op.startswith("experts"):
        k, n, e, m = case["n_in"], case["n_out"], case["experts"], 2 if "gated" in op else 1
        s["perm"], s["offsets"], _, p = _route(case, gen, dev)
        s["x"] = normal(p, k)
        s["w"] = [torch.empty((e, n, k), dtype=dt, device=dev) for _ in range(m)]
        for w in s["w"]:
            for i in range(0, e, 64):
                w[i:i + 64] = normal(*w[i:i + 64].shape, scale=1.0 / math.sqrt(k))
        s["bounds"] = s["offsets"].tolist()  # the plain form's loop bounds
        if op.endswith("backward"):
            s["dy"] = normal(p, n, scale=0.1)
            if m == 2:
                s["pre"] = [_grouped(s["x"], w, s["bounds"]).to(dt) for w in s["w"]]
    else:
        h, k = case["width"], case["top_k"]
        yt = torch.float32 if case["y"] == "f32" else dt
        s["perm"], _, s["topk_w"], s["n_rows"] = _route(case, gen, dev)
        s["inv"] = _invert(s["perm"], t * k)
        wide = h + case["x_pad"]
        s["r"] = normal(t, wide, dtype=yt)[:, :h] if case["residual"] else None
        if op == "dispatch_forward":
            s["x"] = normal(t, wide)[:, :h]
        else:
            s["rows"] = normal(s["n_rows"], h)
        if op == "combine_backward":
            s["dy"] = normal(t, wide, scale=0.1, dtype=yt)[:, :h]
    if own:
        _prepare_own(s)
    return s


# ---- the plain forms ------------------------------------------------------------------------------

def _act(name, z):
    """(value, derivative)"""
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name in ("silu", "sigmoid"):
        p = 1.0 / (1.0 + torch.exp(-z))
        return (p, p * (1.0 - p)) if name == "sigmoid" else (z * p, p * (1.0 + z * (1.0 - p)))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * (1.0 / math.sqrt(2.0))))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _grouped(x, w, bounds):
    """x_r W_e^T in 32 bits, a product for each expert that has rows."""
    out = torch.empty((x.shape[0], w.shape[1]), dtype=torch.float32, device=x.device)
    for e in range(w.shape[0]):
        if bounds[e] < bounds[e + 1]:
            torch.mm(x[bounds[e]:bounds[e + 1]].float(), w[e].float().t(), out=out[bounds[e]:bounds[e + 1]])
    return out


def _grouped_grads(x, w, dy, bounds):
    """(dx in 32 bits, dW rounded) of such a product; dy in 32 bits."""
    dx, dw = torch.empty(x.shape, dtype=torch.float32, device=x.device), torch.zeros_like(w)
    for e in range(w.shape[0]):
        if bounds[e] < bounds[e + 1]:
            rows = slice(bounds[e], bounds[e + 1])
            torch.mm(dy[rows], w[e].float(), out=dx[rows])
            dw[e] = dy[rows].t() @ x[rows].float()
    return dx, dw


def _loss32(x, w, targets):
    z = x.float() @ w.float().t()
    live = targets != IGNORE
    at = torch.where(live, targets, torch.zeros_like(targets)).long()[:, None]
    top = z.max(dim=1, keepdim=True).values
    # the target's own term apart, so that a sure token's small loss keeps its digits
    zt = z.gather(1, at)
    e = torch.exp(z - top).scatter(1, at, 0.0)
    rest = e.sum(dim=1, keepdim=True)
    loss = torch.where(zt == top, torch.log1p(rest), torch.log(rest + torch.exp(zt - top)) + (top - zt))
    lse = loss + zt
    zero = torch.zeros((), device=z.device)
    return torch.where(live, loss[:, 0], zero), torch.where(live, lse[:, 0], zero)


def run(state):
    if own:
        return _run_own(state)
    case, op = state["case"], state["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op.startswith("loss"):
        x, w, targets = state["x"], state["w"], state["targets"]
        if op == "loss_forward":
            loss, lse = _loss32(x, w, targets)
            return {"loss": loss, "lse": lse}
        live = targets != IGNORE
        at = torch.where(live, targets, torch.zeros_like(targets)).long()[:, None]
        wf = w.float()
        dz = torch.exp(x.float() @ wf.t() - state["lse"][:, None])
        dz.scatter_(1, at, torch.expm1(-state["loss"])[:, None])
        dz = torch.where(live[:, None], dz * state["dloss"][:, None], torch.zeros((), device=x.device))
        return {"dx": (dz @ wf).to(dt), "dw": (dz.t() @ x.float()).to(dt)}
    if op.startswith("experts"):
        x, w, bounds = state["x"], state["w"], state["bounds"]
        if op == "experts_linear_forward":
            return {"y": _grouped(x, w[0], bounds).to(dt)}
        if op == "experts_gated_forward":
            g, u = _grouped(x, w[0], bounds), _grouped(x, w[1], bounds)
            out = {"h": (_act(case["act"], g)[0] * u).to(dt)}
            if case["save"]:
                out["gate"], out["up"] = g.to(dt), u.to(dt)
            return out
        dy = state["dy"].float()
        if op == "experts_linear_backward":
            dx, dw = _grouped_grads(x, w[0], dy, bounds)
            return {"dx": dx.to(dt), "dw": [dw]}
        value, slope = _act(case["act"], state["pre"][0].float())
        dxg, dwg = _grouped_grads(x, w[0], dy * state["pre"][1].float() * slope, bounds)
        dxu, dwu = _grouped_grads(x, w[1], dy * value, bounds)
        return {"dx": (dxg + dxu).to(dt), "dw": [dwg, dwu]}
    t, k, h, perm = case["tokens"], case["top_k"], case["width"], state["perm"]
    zero = torch.zeros((), device=perm.device)
    row_pair = perm.clamp(min=0).long()
    if op == "dispatch_forward":
        xs = torch.where(perm[:, None] >= 0, state["x"][row_pair // k].float(), zero)
        return {"xs": xs.to(dt), "inv": _invert(perm, t * k)}
    inv, rows = state["inv"], state["rows"]
    taken = torch.where(inv[:, None] >= 0, rows[inv.clamp(min=0).long()].float(), zero).view(t, k, h)
    if op == "combine_backward":
        dy = state["dy"].float()
        dys = torch.where(perm[:, None] >= 0, state["topk_w"].reshape(-1)[row_pair][:, None] * dy[row_pair // k], zero)
        return {"dys": dys.to(dt), "dw": (taken * dy[:, None, :]).sum(dim=2)}
    if op == "combine_forward":
        taken = taken * state["topk_w"][:, :, None]
    y = taken.sum(dim=1)
    if state["r"] is not None:
        y = y + state["r"].float()
    return {"y": y if case["y"] == "f32" else y.to(dt)}


# ---- the library's entry points -------------------------------------------------------------------

def _prepare_own(s):
    """The plan, the workspace and the outputs that a program keeps."""
    from mixture_experts_route_amd import native as N

    case, op, t = s["case"], s["case"]["op"], s["case"]["tokens"]
    dt, dev = DTYPES[case["dtype"]], torch.device("cuda", torch.cuda.current_device())
    code = N.MOE_BF16 if dt == torch.bfloat16 else N.MOE_F16
    backward = op.endswith("backward")

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev)

    if op.startswith("loss"):
        k, v = case["n_in"], case["vocab"]
        s["d"] = N.loss_dims(k, v, code, IGNORE)
        nbytes = N.moe_loss_workspace_bytes(s["d"], t, backward)
        if backward:
            s["out"] = {"dx": empty(t, k), "dw": empty(v, k)}
        else:
            s["out"] = {"loss": empty(t, dtype=torch.float32), "lse": empty(t, dtype=torch.float32)}
    elif op.startswith("experts"):
        k, n, e, p = case["n_in"], case["n_out"], case["experts"], s["x"].shape[0]
        s["d"] = N.experts_dims(e, k, n, code, getattr(N, "MOE_ACT_" + case["act"].upper()))
        nbytes = N.moe_experts_workspace_bytes(s["d"], p, backward)
        if backward:
            s["out"] = {"dx": empty(p, k), "dw": [empty(e, n, k) for _ in s["w"]]}
        elif op == "experts_linear_forward":
            s["out"] = {"y": empty(p, n)}
        else:
            s["out"] = {"h": empty(p, n)}
            if case["save"]:
                s["out"].update(gate=empty(p, n), up=empty(p, n))
    else:
        h, k, p = case["width"], case["top_k"], s["n_rows"]
        s["d"] = N.rows_dims(h, k, code)
        nbytes = N.moe_rows_workspace_bytes(s["d"], t)
        if op == "dispatch_forward":
            s["out"] = {"xs": empty(p, h), "inv": empty(t * k, dtype=torch.int32)}
        elif op == "combine_backward":
            s["out"] = {"dys": empty(p, h), "dw": empty(t, k, dtype=torch.float32)}
        else:
            s["out"] = {"y": empty(t, h, dtype=torch.float32 if case["y"] == "f32" else dt)}
    s["ws"] = torch.empty((nbytes + 3) // 4, dtype=torch.int32, device=dev)
    N.moe_workspace_init(s["ws"])


def _run_own(s):
    from mixture_experts_route_amd import native as N

    op, t, d, ws, out = s["case"]["op"], s["case"]["tokens"], s["d"], s["ws"], s["out"]
    if op == "dispatch_forward":
        N.moe_dispatch_forward(d, s["x"], t, s["perm"], out["xs"], out["inv"], ws)
    elif op == "dispatch_backward":
        N.moe_dispatch_backward(d, s["rows"], s["inv"], t, out["y"], ws, residual=s["r"])
    elif op == "combine_forward":
        N.moe_combine_forward(d, s["rows"], s["inv"], s["topk_w"], t, out["y"], ws, residual=s["r"])
    elif op == "combine_backward":
        N.moe_combine_backward(d, s["dy"], t, s["perm"], s["inv"], s["topk_w"], ws, ys=s["rows"], dys=out["dys"],
                               dtopk_w=out["dw"])
    elif op == "experts_linear_forward":
        N.moe_experts_linear_forward(d, s["x"], s["offsets"], s["w"][0], out["y"], ws)
    elif op == "experts_gated_forward":
        N.moe_experts_gated_forward(d, s["x"], s["offsets"], s["w"][0], s["w"][1], out["h"], ws, gate=out.get("gate"),
                                    up=out.get("up"))
    elif op == "experts_linear_backward":
        N.moe_experts_linear_backward(d, s["x"], s["offsets"], s["w"][0], s["dy"], ws, dx=out["dx"], dw=out["dw"][0])
    elif op == "experts_gated_backward":
        N.moe_experts_gated_backward(d, s["x"], s["offsets"], s["w"][0], s["w"][1], s["pre"][0], s["pre"][1], s["dy"], ws,
                                     dx=out["dx"], dw_gate=out["dw"][0], dw_up=out["dw"][1])
    elif op == "loss_forward":
        N.moe_loss_forward(d, s["x"], t, s["w"], s["targets"], out["loss"], out["lse"], ws)
    else:
        N.moe_loss_backward(d, s["x"], t, s["w"], s["targets"], s["loss"], s["lse"], s["dloss"], ws, dx=out["dx"],
                            dw=out["dw"])
    return out


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _exact_act(name, z):
    one = torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0.0), torch.heaviside(z, 0.0 * one)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2.0) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(8.0 / math.pi)  # (1 + tanh(v)) / 2 = expit(2 v)
        p = torch.special.expit(a * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1.0 - p) * a * (1.0 + 0.134145 * z.square())
    p, q = torch.special.expit(z), torch.special.expit(-z)
    return (p, p * q) if name == "sigmoid" else (z * p, p + z * p * q)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("loss"):
        x, w = s["x"].double(), s["w"].double()
        z = torch.matmul(x, w.T)
        live = torch.nonzero(s["targets"] != IGNORE)[:, 0]
        hit = s["targets"][live].long()
        if op == "loss_forward":
            loss, lse = torch.zeros_like(z[:, 0]), torch.zeros_like(z[:, 0])
            lse[live] = torch.logsumexp(z[live], dim=1)
            loss[live] = torch.logsumexp(z[live] - z[live, hit][:, None], dim=1)
            return {"loss": loss, "lse": lse}
        p = torch.zeros_like(z)
        p[live] = torch.softmax(z[live], dim=1)
        p[live, hit] -= 1.0
        p.mul_(s["dloss"].double()[:, None])
        return {"dx": torch.matmul(p, w), "dw": torch.matmul(p.T, x)}
    if op.startswith("experts"):
        counts = s["offsets"].diff().tolist()
        xs = [v.double() for v in s["x"].split(counts)]
        per = list(range(case["experts"]))
        if op.endswith("forward"):
            z = [torch.cat([torch.matmul(xs[e], w[e].double().T) for e in per]) for w in s["w"]]
            if len(z) == 1:
                return {"y": z[0]}
            out = {"h": _exact_act(case["act"], z[0])[0].mul(z[1])}
            if case["save"]:
                out.update(gate=z[0], up=z[1])
            return out
        dz = [s["dy"].double()]
        if op == "experts_gated_backward":
            a, da = _exact_act(case["act"], s["pre"][0].double())
            dz = [da.mul_(s["pre"][1].double()).mul_(dz[0]), a.mul_(dz[0])]
        dz = [v.split(counts) for v in dz]
        dx = torch.cat([sum(torch.matmul(v[e], w[e].double()) for v, w in zip(dz, s["w"])) for e in per])
        return {"dx": dx, "dw": [torch.stack([torch.matmul(v[e].T, xs[e]) for e in per]) for v in dz]}
    t, k = case["tokens"], case["top_k"]
    rows = torch.nonzero(s["perm"] >= 0)[:, 0]
    pairs = s["perm"][rows].long()
    tokens = torch.div(pairs, k, rounding_mode="floor")
    if op == "dispatch_forward":
        xs = torch.zeros((s["n_rows"], case["width"]), dtype=torch.float64, device=rows.device)
        xs[rows] = s["x"].double()[tokens]
        inv = torch.full((t * k,), -1, dtype=torch.int32, device=rows.device)
        inv[pairs] = rows.to(torch.int32)
        return {"xs": xs, "inv": inv}
    vals = s["rows"].double()[rows]
    w = s["topk_w"].double().flatten()[pairs]
    if op == "combine_backward":
        dy = s["dy"].double()[tokens]
        dys = torch.zeros((s["n_rows"], case["width"]), dtype=torch.float64, device=rows.device)
        dys[rows] = dy.mul(w[:, None])
        dw = torch.zeros(t * k, dtype=torch.float64, device=rows.device)
        dw[pairs] = vals.mul(dy).sum(1)
        return {"dys": dys, "dw": dw.view(t, k)}
    if op == "combine_forward":
        vals = vals.mul(w[:, None])
    y = torch.zeros((t, case["width"]), dtype=torch.float64, device=rows.device) if s["r"] is None else s["r"].double().clone()
    return {"y": y.index_add_(0, tokens, vals)}
