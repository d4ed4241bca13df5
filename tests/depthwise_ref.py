"""The depthwise layer's backward pass (groups = offset_groups = C) in 64 bits, from fp32
positions, with bounds on what an fp32 computation of it may be off by at every element.

Bounds.  u = 2^-24.  Written for a tap with the neighbours x0 and x1, d = mask w grad_out:
 * grad_offsets = mask w grad_out (x1 - x0) and grad_mask = w grad_out ((1-f) x0 + f x1): four
   roundings, each relative to the product with |x0| + |x1|; 5 u of it covers second orders.
 * grad_x: a contribution is off by at most 6 u |d| (two products for d, one for f d, one
   difference).  An fp32 sum of n contributions adds at most n u sum|d|, an integer sum whose
   unit is at most 2^-22 of the site's largest contribution n 2^-23 sum|d| = 2 n u sum|d| and
   one rounding at its end.  Together (2 n + 8) u sum|d|.
 * grad_weight, grad_bias: chains of at most Lo / 32 + B + 40 additions.
Then the rounding to the type: half a step of the value and of its error.
"""
import torch

import norm_ref as R


def backward(x, off, mask, w, gout, stride, padding, dilation, unconstrained):
    """(gradients, bounds, what each site of grad_x got: sum|d|) as float64 dicts by name;
    x, off, mask (or None), w [C, 1, K] and gout as the library takes them, on any device."""
    B, C, L = x.shape
    Lo, K = off.shape[2:]
    T = gout.dtype
    start = torch.arange(Lo, device=x.device) * stride - padding
    base = (start[:, None] + torch.arange(K, device=x.device) * dilation).float()
    raw = base + off.float()
    pos = raw
    if not unconstrained:
        lo = start.float()[:, None]
        pos = torch.minimum(torch.maximum(raw, lo), lo + float(dilation * (K - 1)))
    i0 = pos.floor()
    f = (pos - i0).double()
    x64, g = x.double(), gout.double()[..., None]
    m = torch.ones_like(f) if mask is None else mask.double()
    dv = w.double().view(1, C, 1, K) * g
    d = m * dv

    def site(i):
        inside = (i >= 0) & (i <= L - 1)
        return torch.where(inside, i, 0.0).long().flatten(2), inside

    at0, in0 = site(i0)
    at1, in1 = site(i0 + 1)
    x0 = torch.where(in0, x64.gather(2, at0).view_as(f), 0.0)
    x1 = torch.where(in1, x64.gather(2, at1).view_as(f), 0.0)
    v = (1 - f) * x0 + f * x1
    inside = (pos == raw).double()
    ref = {"offsets": (x1 - x0) * d * inside, "mask": v * dv, "weight": (m * v * g).sum((0, 2))[:, None],
           "bias": g.sum((0, 2, 3))}
    gx, size, count = (torch.zeros(B, C, L, dtype=torch.float64, device=x.device) for _ in range(3))
    for at, ok, part in ((at0, in0, (1 - f) * d), (at1, in1, f * d)):
        gx.scatter_add_(2, at, torch.where(ok, part, 0.0).flatten(2))
        size.scatter_add_(2, at, torch.where(ok, d.abs(), 0.0).flatten(2))
        count.scatter_add_(2, at, ok.double().flatten(2))
    ref["x"] = gx
    u, h, tiny = R.U, R.half_step(T), torch.finfo(T).tiny
    xs = x0.abs() + x1.abs()
    chain = (Lo / 32 + B + 40) * u * 1.01
    e = {"offsets": 5 * u * xs * d.abs(), "mask": 5 * u * xs * dv.abs(), "x": (2 * count + 8) * u * size,
         "weight": (chain + 8 * u) * (g * m).abs().mul(xs).sum((0, 2))[:, None],
         "bias": chain * g.abs().sum((0, 2, 3))}
    bound = {n: e[n] + h * (ref[n].abs() + e[n]) + tiny for n in ref}
    if mask is None:
        ref.pop("mask"), bound.pop("mask")
    return ref, bound, size
