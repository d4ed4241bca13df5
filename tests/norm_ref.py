"""Plain 64-bit forms of layer norm over the channels and of the 8-bit checkpoint, and the
error bounds of an fp32 computation of them, shared by the CPU and GPU tests.

Bounds.  u = 2^-24 is half a step of fp32; a type T rounds with u_T = finfo(T).eps / 2.  A
sum of n terms added in chains of at most m additions is off by at most m u sum|terms| (to
first order; the factor 1.01 covers the rest).  A kernel adds C channels with at least eight
partial sums and joins them, so m = C / 8 + 40.
"""
import torch

U = 2.0 ** -24
BLOCK = 32


def half_step(t):
    return torch.finfo(t).eps / 2


def norm(x, gamma, beta, eps):
    """y, mean, rstd, v in float64; mean and rstd [B, L]."""
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / (d.square().mean(1) + eps).sqrt()
    v = d * rstd[:, None]
    y = v if gamma is None else v * gamma.double()[:, None]
    y = y if beta is None else y + beta.double()[:, None]
    return y, mean, rstd, v


def norm_bounds(x, gamma, beta, eps):
    """Bounds on |error| of mean, rstd (absolute) and of v, before any rounding to a type."""
    C = x.shape[1]
    m = (C / 8 + 40) * 1.01
    _, mean, rstd, v = norm(x, None, None, eps)
    e_mean = m * U * x.double().abs().mean(1)
    # the second pass squares x - mean' : its sum is off by C (mean' - mean)^2 from the shift,
    # and by (m + 3) u of itself from the differences, products and additions
    var_rel = (m + 6) * U + (e_mean * rstd) ** 2
    e_rstd = rstd * (var_rel / 2 + 4 * U) * 1.01
    e_v = (e_mean * rstd)[:, None] * 1.01 + v.abs() * (e_rstd / rstd + 3 * U)[:, None]
    return e_mean + U * mean.abs(), e_rstd, e_v


def y_bound(y, v, e_v, gamma, T):
    g = 1.0 if gamma is None else gamma.double().abs()[:, None]
    e = g * e_v + 3 * U * (g * v.abs() + y.abs())
    return e * 1.01 + half_step(T) * (y.abs() + e) + torch.finfo(T).tiny


def norm_grads(v, rstd, gamma, gy):
    """grad_x, grad_gamma, grad_beta in float64 from float64 v and rstd."""
    gy = gy.double()
    d = gy if gamma is None else gy * gamma.double()[:, None]
    a, s = d.mean(1, keepdim=True), (d * v).mean(1, keepdim=True)
    gx = rstd[:, None] * (d - a - v * s)
    return {"x": gx, "gamma": (gy * v).sum((0, 2)), "beta": gy.sum((0, 2))}


def grad_bounds(v, e_v, rstd, gamma, gy, T):
    """Bounds on |error| of the three gradients, their final rounding to T included; e_v is
    what the kernel's own v may be off by."""
    B, C, L = gy.shape
    gy = gy.double()
    m = (C / 8 + 40) * 1.01
    d = (gy if gamma is None else gy * gamma.double()[:, None]).abs()
    a, s = d.mean(1, keepdim=True), (d * v.abs()).mean(1, keepdim=True)
    e_a = (m + 2) * U * a
    e_s = (m + 3) * U * s + (d * e_v).mean(1, keepdim=True)
    e = rstd[:, None] * (e_a + v.abs() * e_s + e_v * (s + e_s)
                         + 6 * U * (d + a + v.abs() * s)) * 1.01
    ref = norm_grads(v, rstd, gamma, gy)
    h = half_step(T)
    # weight gradients: B L terms, in chains of at most min(B L, 1500) + 40 additions
    w = (min(B * L, 1500) + 40) * U * 1.01
    e_g = w * (gy * v).abs().sum((0, 2)) + (gy.abs() * e_v).sum((0, 2))
    e_b = w * gy.abs().sum((0, 2))
    tiny = torch.finfo(T).tiny
    return {"x": e + h * (ref["x"].abs() + e) + tiny,
            "gamma": e_g + h * (ref["gamma"].abs() + e_g) + tiny,
            "beta": e_b + h * (ref["beta"].abs() + e_b) + tiny}


def rows_of(t):
    """[rows, n]: the checkpoint's rows (positions of a channel; channels when L == 1)."""
    return t.reshape(t.shape[0], -1) if t.shape[2] == 1 else t.flatten(0, 1)


def step_exponent(amax, top):
    """Exponent of the step of a block whose largest magnitude is amax (float64, finite)."""
    frac, e = torch.frexp(amax.clamp(min=2.0 ** -200))  # amax = frac 2^e, frac in [1/2, 1)
    e = e - 7 + (torch.round(frac * 128) > 127).int()  # the smallest with a code <= 127
    return e.clamp(-126, top)


def two_to(e):
    """2^e exactly (float64) for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pack(x):
    """(codes, scales) of x [B, C, L] in the shapes of the library, from float64."""
    top = 9 if x.dtype == torch.float16 else 121
    r = rows_of(x.double())
    n = r.shape[1]
    blocks = torch.nn.functional.pad(r, (0, -n % BLOCK)).unflatten(1, (-1, BLOCK))
    amax = blocks.abs().amax(2)
    bad = ~torch.isfinite(amax)
    e = step_exponent(torch.where(bad, 1.0, amax), top)
    codes = torch.round(torch.where(bad[..., None], 0.0, blocks) / two_to(e)[..., None])
    codes = codes.clamp(-127, 127).flatten(1)[:, :n].to(torch.int8).reshape(x.shape)
    scales = torch.where(bad, 255, e + 127).to(torch.uint8)
    B, C, L = x.shape
    return codes, scales.reshape((B, -1, 1) if L == 1 else (B, C, -1))


def values(codes, scales):
    """What a checkpoint stands for, float64."""
    r = rows_of(codes).double()
    n = r.shape[1]
    s = scales.reshape(r.shape[0], -1).int()
    step = torch.where(s == 255, float("nan"), two_to(s - 127))
    return (r * step.repeat_interleave(BLOCK, 1)[:, :n]).reshape(codes.shape)
