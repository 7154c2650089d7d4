"""The linear layer and layer norm in 64 bits on the CPU, with error bounds.

Each function returns (exact values, bound on a kernel's distance from them).
The bounds count roundings: u = 2^-24 for each binary32 operation (2^-23 for
a sum inside the matrix units, which may cut instead of round), half a step
of the output's type for the last rounding, and half a step for dz, which is
rounded before the gradients' products.
"""

import math

import torch

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(t):
    return torch.finfo(t).eps / 2


def rounded(exact, before, t):
    """Bound after one rounding to t of a value that is `before` off."""
    size = exact.abs() + before
    return before + half_step(t) * size + torch.finfo(t).smallest_normal * half_step(t)


def activate(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# Error of an activation or of its slope as the kernels evaluate them, apart
# from the error of z: the fast forms' erfc is 1.5e-7 off, their exp2 takes an
# argument with a relative error of 2u (|z| up to 12 matters: beyond, the
# result is 0 or z to all bits), and some ten operations of u each follow.
def act_error(z):
    return (1.5e-7 + 64 * U) * (1 + z.abs())


def product(a, b):
    """a @ b.T in 64 bits and the bound of its sums in the matrix units."""
    a, b = a.double(), b.double()
    return a @ b.t(), (a.shape[1] + 4) * 2 * U * (a.abs() @ b.abs().t())


def linear(x, w, bias, residual, act):
    t = x.dtype
    z, dz = product(x, w)
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2 * U * z.abs()
    y = activate(z, act)
    dy = 1.2 * dz + (act_error(z) if act != "none" else 0.0)  # slopes are at most 1.13
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2 * U * (y.abs() + residual.double().abs())
    return (y, rounded(y, dy, t)), (z, rounded(z, dz, t))


def linear_backward(dy, x, w, z, act):
    t = dy.dtype
    g = dy.double()
    off = torch.zeros_like(g)  # of dz as the products use it
    near = torch.zeros_like(g)  # of dz as the bias gradient sums it
    if act != "none":
        s = slope(z.double(), act)
        near = g.abs() * ((act_error(z.double()) if act != "relu" else 0.0) + 2 * U * s.abs())
        g = g * s
        off = rounded(g, near, t)
    dx, ex = product(g, w.t())
    dw, ew = product(g.t(), x.t())
    ex = ex * 1.01 + off @ w.double().abs()
    ew = ew * 1.01 + off.t() @ x.double().abs()
    db = g.sum(0)
    eb = near.sum(0) + (dy.shape[0] + 4) * U * (g.abs() + near).sum(0)
    return (dx, rounded(dx, ex, t)), (dw, rounded(dw, ew, t)), (db, rounded(db, eb, t))


def _sum_error(width):
    """Relative to the sum of sizes: a thread adds up to width / 64 values (or, with more threads, fewer), a tree the rest."""
    return (min(width, width // 64 + 24) + 2) * U


def layer_norm(x, w, b, eps):
    t = x.dtype
    v = x.double()
    n = v.shape[1]
    mean = v.mean(1, keepdim=True)
    d = v - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    h = d * rstd
    off_mean = (_sum_error(n) + U) * v.abs().mean(1, keepdim=True)
    off_d = off_mean + U * (d.abs() + off_mean)
    # the variance: its sum's rounding, and d's error (2 d off_d on average, and its square)
    off_var = (_sum_error(n) + 4 * U) * var + 2 * (d.abs() * off_d).mean(1, keepdim=True) + (off_d ** 2).mean(1, keepdim=True)
    rel = 0.5 * off_var / (var + eps) + 4 * U
    rel = torch.where(rel > 0.25, torch.full_like(rel, math.inf), 1.5 * rel)  # first order holds below that
    off_h = rstd * off_d * (1 + rel) + h.abs() * (rel + 2 * U)
    ww = torch.ones(n, dtype=torch.float64, device=v.device) if w is None else w.double()
    bb = torch.zeros(n, dtype=torch.float64, device=v.device) if b is None else b.double()
    y = h * ww + bb
    off = off_h * ww.abs() + 2 * U * ((h * ww).abs() + bb.abs())
    return ((y, rounded(y, off, t)), (mean[:, 0], off_mean[:, 0] + 2 * U * mean[:, 0].abs()),
            (rstd[:, 0], (rstd * rel)[:, 0]))


def layer_norm_backward(dy, x, mean, rstd, w, param_type):
    t = dy.dtype
    g0, v = dy.double(), x.double()
    n = v.shape[1]
    m, r = mean.double()[:, None], rstd.double()[:, None]
    h = (v - m) * r
    off_h = 2 * U * h.abs()
    ww = torch.ones(n, dtype=torch.float64, device=v.device) if w is None else w.double()
    g = g0 * ww
    off_g = U * g.abs()
    c0, c1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    off0 = (_sum_error(n) + 4 * U) * g.abs().mean(1, keepdim=True)
    off1 = (_sum_error(n) + 8 * U) * (g * h).abs().mean(1, keepdim=True)
    dx = r * (g - c0 - h * c1)
    size = g.abs() + c0.abs() + (h * c1).abs()
    off = r.abs() * (off_g + off0 + h.abs() * off1 + off_h * c1.abs() + 4 * U * size)
    rows = v.shape[0]
    dw = (g0 * h).sum(0)
    ow = ((rows + 8) * U * (g0 * h).abs() + g0.abs() * off_h).sum(0)
    db = g0.sum(0)
    ob = (rows + 8) * U * g0.abs().sum(0)
    return (dx, rounded(dx, off, t)), (dw, rounded(dw, ow, param_type)), (db, rounded(db, ob, param_type))


def assert_within(got, want, name):
    exact, bound = want
    g = got.detach().to(exact.device).double()
    assert g.shape == exact.shape, f"{name}: shape {tuple(g.shape)}"
    assert bool(torch.isfinite(g).all()), f"{name}: not finite"
    over = (g - exact).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{name}: {int((over > 0).sum())} of {over.numel()} values outside their bound, worst by {worst:.3g}"
