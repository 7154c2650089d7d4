"""The gated feed-forward block and the 8-bit products in 64 bits on the CPU (or on the GPU, for
large cases), with error bounds, in the manner of operator_oracle.py.

Each function returns (exact values, bound on a kernel's distance from them).
"""

import torch

import operator_oracle as O
from operator_oracle import U, act_error, activate, product, rounded, slope

LEAST = 2.0 ** -100


def _gate(z, dz, v, dv, act):
    """activate(z) * v for z and v that are dz and dv off."""
    a = activate(z, act)
    da = 1.2 * dz + (act_error(z) if act != "none" else 0.0)  # slopes are at most 1.13
    y = a * v
    off = da * v.abs() + (a.abs() + da) * dv
    return y, off + 2 * U * (y.abs() + off)


def _with_bias(z, dz, bias):
    if bias is None:
        return z, dz
    z = z + bias.double()
    return z, dz + 2 * U * z.abs()


def gated_linear(x, wg, wu, bg, bu, act):
    t = x.dtype
    z, dz = _with_bias(*product(x, wg), bg)
    v, dv = _with_bias(*product(x, wu), bu)
    y, dy = _gate(z, dz, v, dv, act)
    return (y, rounded(y, dy, t)), (z, rounded(z, dz, t)), (v, rounded(v, dv, t))


def gated_linear_backward(dy, x, wg, wu, z, v, act):
    t = dy.dtype
    g, z, v = dy.double(), z.double(), v.double()
    a, s = activate(z, act), slope(z, act)
    inexact = 0.0 if act in ("none", "relu") else act_error(z)
    dz, near_z = g * v * s, (g * v).abs() * (inexact + 4 * U * s.abs())
    dv, near_v = g * a, g.abs() * (inexact + 4 * U * a.abs())
    # what the products take is rounded to the type, what the biases' sums take is not
    off_z, off_v = rounded(dz, near_z, t), rounded(dv, near_v, t)
    (xg, eg), (xu, eu) = product(dz, wg.t()), product(dv, wu.t())
    dx = xg + xu
    # either weight's sums may be rounded once more where the two meet
    ex = (eg + eu) * 1.01 + 4 * U * (xg.abs() + xu.abs()) + off_z @ wg.double().abs() + off_v @ wu.double().abs()
    out = [(dx, rounded(dx, ex, t))]
    for d, off in ((dz, off_z), (dv, off_v)):
        dw, ew = product(d.t(), x.t())
        out.append((dw, rounded(dw, ew * 1.01 + off.t() @ x.double().abs(), t)))
    for d, near in ((dz, near_z), (dv, near_v)):
        eb = near.sum(0) + (dy.shape[0] + 4) * U * (d.abs() + near).sum(0)
        out.append((d.sum(0), rounded(d.sum(0), eb, t)))
    return out


def quantize(x):
    """What the definition gives, bit for bit: every operation is one of binary32, which the CPU rounds as defined."""
    x = x.float()
    size = x.abs().amax(1).clamp(min=LEAST)
    most = torch.full_like(size, 127.0)
    q = torch.round(x * (most / size)[:, None])  # a number over a tensor would be a reciprocal and a product
    return q.to(torch.int8), size / most


def _int8_product(q, scale, w, w_scale):
    z = q.double() @ w.double().t()  # whole numbers below 2^31: exact
    z = z * scale.double()[:, None] * w_scale.double()
    return z, 4 * U * z.abs()  # the sum's rounding and two products'


def linear_quantized(q, scale, w, w_scale, bias, residual, act, t):
    z, dz = _with_bias(*_int8_product(q, scale, w, w_scale), bias)
    y = activate(z, act)
    dy = 1.2 * dz + (act_error(z) if act != "none" else 0.0)
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2 * U * (y.abs() + residual.double().abs())
    return y, rounded(y, dy, t)


def gated_linear_quantized(q, scale, wg, sg, wu, su, bg, bu, act, t):
    z, dz = _with_bias(*_int8_product(q, scale, wg, sg), bg)
    v, dv = _with_bias(*_int8_product(q, scale, wu, su), bu)
    y, dy = _gate(z, dz, v, dv, act)
    return y, rounded(y, dy, t)


assert_within = O.assert_within
