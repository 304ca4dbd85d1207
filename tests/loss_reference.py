"""Softmax cross entropy in float64 with elementwise bounds on what fp32 sums of 16-bit operands may differ by.

Bounds (e = 2^-24, h and d as in dense_reference): a logit's fp32 sum 2 n_in e sum|terms| =: ez; exp by the hardware's exp2
of a rounded argument a: relative (|a| + 4) 2 e; the sum of exponentials through at most 64 + vocab / 512 additions.
  loss   a shift of every other logit against the target's by s moves it by at most (1 - p) (e^s - 1), with s two ez; the
         sum's relative error counts with the same factor; 8 e of the result and of the logits' distance
  lse    ez, the sum's relative error, 8 e of the magnitudes added
  dz     p's relative error is ez's and exp's; at the target expm1's, 8 e; then 2 e for each of: the factor S that dloss is
         multiplied by (1 / the largest |dloss|, fp16 2^11 / it), that product, the one with p, and the results' factor;
         rounded to the type h |dz| + d / S
"""

import torch

import dense_reference as R

E = R.E


def _logits(x, w):
    x, w = x.double(), w.double()
    return x @ w.T, 2 * x.shape[1] * E * (x.abs() @ w.abs().T)


def forward(x, w, targets, ignore):
    z, ez = _logits(x, w)
    V = w.shape[0]
    live = (targets >= 0) & (targets < V) & (targets != ignore)
    at = torch.where(live, targets, 0).long()[:, None]
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, at)
    others = torch.exp(z - zt).scatter(1, at, 0.0).sum(1)
    loss = torch.log1p(others)
    # where that overflows: a distance instead
    loss = torch.where(torch.isinf(loss) & torch.isfinite(lse), lse - zt[:, 0], loss)
    ez = ez.max(1).values
    span = z.max(1).values - z.min(1).values
    r = (span + 4) * 2 * E + (64 + V / 512) * 2 * E
    miss = -torch.expm1(-loss)  # 1 - p
    e_loss = miss * (torch.expm1(2 * ez) + r) + 8 * E * loss
    e_lse = ez + r + 8 * E * (lse.abs() + span)
    zero = torch.zeros_like(loss)
    nan = torch.where(targets == ignore, 0.0, float("nan"))
    out = {}
    for name, v, err in (("loss", loss, e_loss), ("lse", lse, e_lse)):
        out[name] = (torch.where(live, v, nan), torch.where(live, R._round(v, err, torch.float32), zero))
    return out


def dz_of(x, w, targets, ignore, loss, lse, dloss):
    """dz and the bound on the fp32 one."""
    z, ez = _logits(x, w)
    live = (targets >= 0) & (targets < w.shape[0]) & (targets != ignore)
    at = torch.where(live, targets, 0).long()[:, None]
    a = z - lse.double()[:, None]
    p = torch.exp(a)
    ep = p * (torch.expm1(ez) + (a.abs() + 4) * 2 * E)
    own = torch.expm1(-loss.double())[:, None]
    p, ep = p.scatter(1, at, own), ep.scatter(1, at, 8 * E * own.abs())
    g = dloss.double()[:, None]
    dz = torch.where(live[:, None], p * g, 0.0)
    return dz, torch.where(live[:, None], ep * g.abs() + 8 * E * dz.abs(), 0.0)


def backward(x, w, targets, ignore, loss, lse, dloss, dt):
    dz, e = dz_of(x, w, targets, ignore, loss, lse, dloss)
    x, w = x.double(), w.double()
    live = (targets >= 0) & (targets < w.shape[0]) & (targets != ignore)
    most = torch.where(live, dloss.double().abs(), 0.0).max().item()
    tiny = R.tiny_step(dt) * most / (2.0 ** 11 if dt == torch.float16 else 1.0)
    r = e + R.half_step(dt) * (dz.abs() + e) + torch.where(live[:, None], tiny, 0.0)
    out = {}
    for name, a, ra, b in (("dx", dz, r, w), ("dw", dz.T, r.T, x)):
        v = a @ b
        err = ra @ b.abs() + 2 * a.shape[1] * E * ((a.abs() + ra) @ b.abs())
        out[name] = (v, R._round(v, err, dt))
    return out
