"""The dense operators in float64 on plain tensors, with elementwise bounds on what fp32 sums of 16-bit
operands, one rounding of the result and (backward) one rounding of dz may differ by.

Bounds (h = half a step of the type, eps / 2; d = half a step of its smallest numbers, fp16 2^-25;
e = 2^-24 fp32's half step; products of 16-bit operands are exact in fp32):
  a sum of n terms          n e sum|terms| (any order; the matrix cores may chop instead of round: 2 n e)
  an activation             its slope is at most 1.13 and its evaluation is within (6 + |z|) 2 e |z| + 8 e
  its derivative            within 2^-19 (a few fp32 roundings of terms of magnitude up to 2)
  a result of the type      h |v| + d; of fp32: e |v|
  dz rounded to the type    h |dz| + d per term of the products that follow
"""

import math

import torch

E = 2.0 ** -24
NONE, SILU, GELU, GELU_TANH, RELU, SIGMOID = range(6)


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny_step(dt):
    return 2.0 ** -25 if dt == torch.float16 else (2.0 ** -134 if dt == torch.bfloat16 else 2.0 ** -150)


def act(a, z):
    if a == SILU:
        return z * torch.sigmoid(z)
    if a == GELU:
        return z * torch.special.ndtr(z)
    if a == GELU_TANH:
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if a == RELU:
        return torch.relu(z)
    if a == SIGMOID:
        return torch.sigmoid(z)
    return z


def dact(a, z):
    z = z.detach().clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act(a, z).sum(), z)
    return g


def _sum_err(n, mag):
    return 2 * n * E * mag


def _pre(x, w, b):
    """z, and the bound on fp32's z."""
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, mag = z + b, mag + b.abs()
    return z, _sum_err(x.shape[1] + 1, mag)


def _act_err(a, z, ez):
    if a == NONE:
        return z, ez
    return act(a, z), 1.13 * ez + (6 + z.abs()) * 2 * E * z.abs() + 8 * E


def _round(v, err, dt):
    if dt == torch.float32:
        return err + E * (v.abs() + err)
    return err + half_step(dt) * (v.abs() + err) + tiny_step(dt)


def linear_forward(a, x, w, b, r, y_dtype):
    """{name: (value, bound)} for y and pre; x's type is the operands'."""
    dt = x.dtype
    x, w, b, r = (None if t is None else t.double() for t in (x, w, b, r))
    z, ez = _pre(x, w, b)
    y, ey = _act_err(a, z, ez)
    if r is not None:
        y, ey = y + r, ey + E * (y + r).abs() + E * ey
    return {"y": (y, _round(y, ey, y_dtype)), "pre": (z, _round(z, ez, dt))}


def gated_forward(a, x, wg, wu, bg, bu):
    dt = x.dtype
    x, wg, wu, bg, bu = (None if t is None else t.double() for t in (x, wg, wu, bg, bu))
    g, eg = _pre(x, wg, bg)
    u, eu = _pre(x, wu, bu)
    v, ev = _act_err(a, g, eg)
    h = v * u
    eh = ev * (u.abs() + eu) + v.abs() * eu + E * h.abs()
    return {"h": (h, _round(h, eh, dt)), "gate": (g, _round(g, eg, dt)), "up": (u, _round(u, eu, dt))}


def _products(dt, dzs, errs, ws, x):
    """dx, dw, db from the exact dz's and the bounds on the fp32 dz's (before their rounding)."""
    out = {}
    rounded = [e + half_step(dt) * (z.abs() + e) + tiny_step(dt) if e is not None else torch.zeros_like(z)
               for z, e in zip(dzs, errs)]
    n = sum(z.shape[1] for z in dzs)
    dx = sum(z @ w for z, w in zip(dzs, ws))
    mag = sum((z.abs() + r) @ w.abs() for z, r, w in zip(dzs, rounded, ws))
    edx = sum(r @ w.abs() for r, w in zip(rounded, ws)) + _sum_err(n, mag)
    out["dx"] = (dx, _round(dx, edx, dt))
    for i, (z, r, e) in enumerate(zip(dzs, rounded, errs)):
        dw = z.T @ x
        edw = r.T @ x.abs() + _sum_err(z.shape[0], (z.abs() + r).T @ x.abs())
        out[f"dw{i}"] = (dw, _round(dw, edw, dt))
        db = z.sum(0)
        edb = (0 if e is None else e.sum(0)) + _sum_err(z.shape[0], z.abs().sum(0))
        out[f"db{i}"] = (db, _round(db, edb, dt))
    return out


def linear_backward(a, x, w, pre, dy):
    dt = x.dtype
    x, w, dy = x.double(), w.double(), dy.double()
    if a == NONE:
        return _products(dt, [dy], [None], [w], x)
    d = dact(a, pre.double())
    dz = dy * d
    return _products(dt, [dz], [dy.abs() * 2.0 ** -19 + 2 * E * dz.abs()], [w], x)


def gated_backward(a, x, wg, wu, gate, up, dh):
    dt = x.dtype
    x, wg, wu, g, u, dh = (t.double() for t in (x, wg, wu, gate, up, dh))
    v, ev = _act_err(a, g, torch.zeros_like(g))
    d = dact(a, g)
    dg, du = dh * u * d, dh * v
    return _products(dt, [dg, du], [(dh * u).abs() * 2.0 ** -19 + 3 * E * dg.abs(), dh.abs() * ev + 2 * E * du.abs()],
                     [wg, wu], x)


def check(name, got, ref):
    """Every element of ``got`` within its bound of the float64 value."""
    val, bound = ref
    assert got.shape == val.shape, (name, got.shape, val.shape)
    err = (got.double() - val).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int(torch.where(bad.flatten(), err.flatten() / bound.flatten().clamp(min=1e-300), 0.0).nan_to_num(1e300).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{got.flatten()[i].item()}, want {val.flatten()[i].item()} +- {bound.flatten()[i].item()}")
